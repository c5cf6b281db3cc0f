// spans.h -- which bytes a call's matrices take, and whether two of them share some.
#pragma once

#include <algorithm>
#include <cstdint>
#include <initializer_list>

namespace gemmar {

// `rows` rows of `row` bytes, `stride` bytes apart.
struct Span {
    intptr_t at;   // 0: left out
    int64_t row, stride, rows;
};

inline Span span(const void *p, int64_t bytes) { return {reinterpret_cast<intptr_t>(p), bytes, bytes, 1}; }

// A matrix of M rows; stride 0 is one row that stands for all, and rows without a gap are one.
inline Span span_rows(const void *p, int64_t row, int64_t stride, int64_t M)
{
    if (stride == 0 || M == 1)
        return span(p, row);
    return stride == row ? span(p, row * M) : Span{reinterpret_cast<intptr_t>(p), row, stride, M};
}

// Does a row of a meet the n bytes at `at`?
inline bool meets_bytes(const Span &a, intptr_t at, int64_t n)
{
    const int64_t d = at - a.at;
    if (d >= (a.rows - 1) * a.stride + a.row || -d >= n)
        return false;
    return d < 0 || a.rows == 1 || d % a.stride < a.row || a.stride - d % a.stride < n;
}

inline bool meet(const Span &a, const Span &b)
{
    if (a.at == 0 || b.at == 0)
        return false;
    if (b.rows == 1)
        return meets_bytes(a, b.at, b.row);
    if (a.rows == 1)
        return meets_bytes(b, a.at, a.row);
    const int64_t d = b.at - a.at, a_end = (a.rows - 1) * a.stride + a.row, b_end = (b.rows - 1) * b.stride + b.row;
    if (d >= a_end || -d >= b_end)
        return false;
    if (a.stride == b.stride) {   // columns of one wider matrix lie between one another
        const int64_t off = (d % a.stride + a.stride) % a.stride;
        return off < a.row || a.stride - off < b.row;
    }
    // row by row, of those of b that are within a's reach
    for (int64_t i = std::max<int64_t>(0, (-d - b.row) / b.stride); i < b.rows && d + i * b.stride < a_end; ++i)
        if (meets_bytes(a, b.at + i * b.stride, b.row))
            return true;
    return false;
}

// Does an output meet an input or another output?
inline bool any_meet(std::initializer_list<Span> outs, std::initializer_list<Span> ins)
{
    for (const Span *o = outs.begin(); o != outs.end(); ++o) {
        for (const Span *p = o + 1; p != outs.end(); ++p)
            if (meet(*o, *p))
                return true;
        for (const Span &i : ins)
            if (meet(*o, i))
                return true;
    }
    return false;
}

}  // namespace gemmar
