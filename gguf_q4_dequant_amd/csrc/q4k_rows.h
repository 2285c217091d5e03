// Rows of a packed matrix that one buffer covers (plain C++, no device calls:
// also compiled and checked on the host).
#pragma once

namespace q4k {

struct RowWindow {
    int first, rows;
};

// Rows n .. n + most - 1 of a matrix of N rows, N >= 1: those that exist, and
// row N - 1 where none does.  Never empty, because the copies walk along a row
// by the buffer's scalar offset and the hardware's range check compares a
// lane's offset with (size - scalar offset): of a buffer of 0 bytes that
// difference is negative, and where it is taken as unsigned, every lane reads
// from behind the matrix.  With a row or more the scalar offset, less than one
// row, is always below the size.
constexpr RowWindow row_window(int n, int most, int N) {
    const int first = n < N ? n : N - 1;
    return {first, N - first < most ? N - first : most};
}

}  // namespace q4k
