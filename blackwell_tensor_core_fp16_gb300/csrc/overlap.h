// Whether two strided tensors share memory (host only).  The operators refuse a written tensor that
// shares memory with another operand: their blocks read and write in no fixed order.
#pragma once

#include <algorithm>
#include <cstdint>
#include <cstring>
#include <initializer_list>

namespace decode {

// The bytes that a tensor's elements take: a dense run, and up to four strided dimensions around it.
class Footprint {
public:
    // `run`: bytes that are dense in memory; sizes and strides (in bytes) of the dimensions around
    // them.
    template <int N>
    Footprint(const void* base, int64_t run, const int64_t (&sizes)[N], const int64_t (&strides)[N])
        : base_(reinterpret_cast<uintptr_t>(base))
    {
        static_assert(N <= 4, "at most four strided dimensions");
        empty_ = base == nullptr || run <= 0;
        for (int d = 0; d < N; ++d) {
            empty_ = empty_ || sizes[d] <= 0;
            if (sizes[d] > 1 && strides[d] > 0) dim_[dims_++] = {sizes[d], strides[d]};
        }
        std::sort(dim_, dim_ + dims_, [](const Dim& a, const Dim& b) { return a.stride > b.stride; });
        dim_[dims_++] = {run, 1};
        for (int d = dims_ - 2; d >= 0; --d) {           // dimensions that continue each other
            if (dim_[d].stride != dim_[d + 1].size * dim_[d + 1].stride) continue;
            dim_[d + 1].size *= dim_[d].size;
            std::copy(dim_ + d + 1, dim_ + dims_, dim_ + d);
            --dims_;
        }
        for (int d = dims_ - 1; d >= 0; --d)
            span_[d] = (d + 1 < dims_ ? span_[d + 1] : 1) + (dim_[d].size - 1) * dim_[d].stride;
    }
    Footprint(const void* base, int64_t bytes) : Footprint(base, bytes, {1}, {0}) {}

    // True where a byte belongs to both.  Exact, but for layouts whose strides differ and that
    // interleave more than a few thousand times: those count as shared.
    friend bool overlap(const Footprint& a, const Footprint& b)
    {
        if (a.empty_ || b.empty_) return false;
        int budget = 1 << 14;
        return meet(a, 0, b, 0, static_cast<int64_t>(b.base_ - a.base_), budget);
    }

private:
    struct Dim {
        int64_t size, stride;
    };
    // a's dimensions from x on and b's from y on, whose origin lies `delta` bytes behind a's
    static bool meet(const Footprint& a, int x, const Footprint& b, int y, int64_t delta, int& budget)
    {
        if (delta >= a.span_[x] || -delta >= b.span_[y]) return false;
        const bool run_a = x + 1 == a.dims_, run_b = y + 1 == b.dims_;
        if ((run_a && run_b) || --budget < 0) return true;
        const Dim &p = a.dim_[x], &q = b.dim_[y];
        if (!run_a && !run_b && p.stride == q.stride && a.span_[x + 1] <= p.stride &&
            b.span_[y + 1] <= p.stride) {
            // only the difference m of the two indices matters, and few m bring the rests together
            const int64_t s = p.stride;
            const int64_t lo = std::max(1 - p.size, floor_div(-b.span_[y + 1] - delta, s));
            const int64_t hi = std::min(q.size - 1, floor_div(a.span_[x + 1] - delta, s));
            for (int64_t m = lo; m <= hi; ++m)
                if (meet(a, x + 1, b, y + 1, delta + m * s, budget)) return true;
            return false;
        }
        if (run_b || (!run_a && p.stride >= q.stride)) {     // those of a's rests that b's span reaches
            const int64_t lo = std::max<int64_t>(0, floor_div(delta - a.span_[x + 1], p.stride));
            const int64_t hi = std::min(p.size - 1, floor_div(delta + b.span_[y], p.stride));
            for (int64_t i = lo; i <= hi; ++i)
                if (meet(a, x + 1, b, y, delta - i * p.stride, budget)) return true;
            return false;
        }
        const int64_t lo = std::max<int64_t>(0, floor_div(-delta - b.span_[y + 1], q.stride));
        const int64_t hi = std::min(q.size - 1, floor_div(a.span_[x] - delta, q.stride));
        for (int64_t j = lo; j <= hi; ++j)
            if (meet(a, x, b, y + 1, delta + j * q.stride, budget)) return true;
        return false;
    }
    static int64_t floor_div(int64_t a, int64_t b) { return a / b - (a % b < 0 ? 1 : 0); }

    uintptr_t base_;
    Dim dim_[5] = {};
    int64_t span_[5] = {};                 // bytes from the first to the last of dimensions d, d + 1, ...
    int dims_ = 0;
    bool empty_ = false;
};

// An operand of a call: up to three strided dimensions (strides in elements) around rows of `row`
// dense elements of `bytes` bytes each.
class Operand {
public:
    template <int N>
    Operand(const char* name, const void* base, int64_t bytes, int64_t row, const int64_t (&sizes)[N],
            const int64_t (&strides)[N], const char* may_be = nullptr)
        : name(name), may_be(may_be), base_(base), run_(row * bytes)
    {
        static_assert(N <= 3, "at most three strided dimensions");
        int64_t last = run_;
        bool empty = base == nullptr || row <= 0;
        for (int d = 0; d < N; ++d) {
            empty = empty || sizes[d] <= 0;
            size_[d] = sizes[d];
            stride_[d] = sizes[d] > 1 ? strides[d] * bytes : 0;
            last += (size_[d] - 1) * stride_[d];
        }
        first_ = empty ? 0 : reinterpret_cast<uintptr_t>(base);
        end_ = empty ? 0 : first_ + static_cast<uintptr_t>(last);
    }
    Operand(const char* name, const void* base, int64_t bytes, int64_t count)
        : Operand(name, base, bytes, count, {1}, {0})
    {
    }
    const char* name;
    const char* may_be;      // a written operand: the name of the input that it may be itself

    friend bool overlap(const Operand& a, const Operand& b)
    {
        // (almost always decided here)
        if (a.end_ <= b.first_ || b.end_ <= a.first_) return false;
        return overlap(a.footprint(), b.footprint());
    }
    friend bool same(const Operand& a, const Operand& b)
    {
        return a.base_ == b.base_ && a.run_ == b.run_ && std::equal(a.size_, a.size_ + 3, b.size_) &&
               std::equal(a.stride_, a.stride_ + 3, b.stride_);
    }

private:
    Footprint footprint() const { return Footprint(base_, run_, size_, stride_); }
    const void* base_;
    int64_t run_;
    int64_t size_[3] = {1, 1, 1}, stride_[3] = {0, 0, 0};   // of one element: stride 0; in bytes
    uintptr_t first_, end_;
};

// The first written operand that shares memory with another operand, and that one; false if none
// does.
inline bool find_shared(std::initializer_list<Operand> written, std::initializer_list<Operand> read,
                        const char*& one, const char*& other)
{
    const auto is = [](const char* a, const char* b) { return a != nullptr && !std::strcmp(a, b); };
    for (const Operand& w : written) {
        one = w.name;
        for (const Operand& r : read) {
            other = r.name;
            if (overlap(w, r) && !(is(w.may_be, r.name) && same(w, r))) return true;
        }
        for (const Operand& x : written) {
            if (&x == &w) break;
            other = x.name;
            if (overlap(w, x)) return true;
        }
    }
    return false;
}

}  // namespace decode
