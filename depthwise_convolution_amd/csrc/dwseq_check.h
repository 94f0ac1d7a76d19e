// dwseq_check.h -- the checks of arguments that the C entry points of the sequence
// and mixing operators share.  Plain C++.
#pragma once

#include "../../include/dwconv_seq.h"
#include "dwseq_internal.h"

#include <cstdint>

namespace dwseq {

// An array of `rows` rows of `width` bytes, `ld` bytes from row to row.
struct Region {
    std::uintptr_t base;
    long long rows, ld, width;
    bool empty() const { return base == 0 || rows <= 0 || width <= 0; }
    std::uintptr_t end() const
    {
        return base + static_cast<std::uintptr_t>((rows - 1) * ld + width);
    }
};

inline Region region(const void *p, long long rows, long long ld, long long width)
{
    return Region{reinterpret_cast<std::uintptr_t>(p), rows, ld, width};
}

inline Region dense(const void *p, long long bytes) { return region(p, 1, bytes, bytes); }

// Whether two arrays share a byte.  Column ranges of one wider array (equal
// row strides) are told apart; other arrays by their extent alone.
inline bool overlap(const Region &a, const Region &b)
{
    if (a.empty() || b.empty() || a.base >= b.end() || b.base >= a.end())
        return false;
    if (a.ld != b.ld || (a.rows == 1 && b.rows == 1))
        return true;
    const Region &lo = a.base <= b.base ? a : b, &hi = a.base <= b.base ? b : a;
    const long long d = static_cast<long long>((hi.base - lo.base) % lo.ld);
    return !(d >= lo.width && d + hi.width <= lo.ld);
}

inline bool aligned(const void *p, int to) { return (reinterpret_cast<std::uintptr_t>(p) % to) == 0; }

// Collects the arrays of a call and what is wrong with them.
class Check {
  public:
    int status = DWCONV_OK;

    void fail(int code)
    {
        if (status == DWCONV_OK)
            status = code;
    }
    // an input that the call may write over, in place: it is listed as an output only
    void check(const void *p, const Region &r, int align) { array(p, r, align, true); }
    // must: the pointer may not be NULL (when the array has any row)
    void in(const void *p, const Region &r, int align, bool must = true)
    {
        array(p, r, align, must);
        if (!r.empty() && n_in < kMost)
            ins[n_in++] = r;
    }
    void out(const void *p, const Region &r, int align, bool must = true)
    {
        array(p, r, align, must);
        if (r.empty())
            return;
        for (int k = 0; k < n_out; ++k)
            if (overlap(outs[k], r))
                clash = true;
        if (n_out < kMost)
            outs[n_out++] = r;
    }
    int done()
    {
        for (int o = 0; o < n_out; ++o)
            for (int k = 0; k < n_in; ++k)
                if (overlap(outs[o], ins[k]))
                    clash = true;
        if (clash)
            fail(DWCONV_ERR_ALIAS);
        return status;
    }

  private:
    static constexpr int kMost = 16;
    Region ins[kMost], outs[kMost];
    int n_in = 0, n_out = 0;
    bool clash = false;

    void array(const void *p, const Region &r, int align, bool must)
    {
        if (!p && must && r.rows > 0)
            fail(DWCONV_ERR_NULL_PTR);
        if (p && !aligned(p, align))
            fail(DWCONV_ERR_MISALIGNED);
    }
};

inline bool type_ok(int type) { return type >= DWCONV_T_F32 && type <= DWCONV_T_BF16; }
inline bool act_ok(int act) { return act >= DWCONV_ACT_NONE && act <= DWCONV_ACT_SILU; }

// Rows of a batch: DWCONV_OK and *b, or what is wrong.
inline int make_batch(int seqs, long long tokens, const int *offsets, bool packed, Batch *b)
{
    if (seqs < 1 || seqs > DWCONV_SEQ_MAX_ROWS || tokens < 0 || tokens > DWCONV_SEQ_MAX_ROWS)
        return DWCONV_ERR_BAD_DIM;
    const long long rows = packed ? tokens : tokens * seqs;
    if (rows > DWCONV_SEQ_MAX_ROWS)
        return DWCONV_ERR_BAD_DIM;
    if (offsets && !aligned(offsets, 4))
        return DWCONV_ERR_MISALIGNED;
    b->seqs = seqs;
    b->rows = (int)rows;
    b->tokens = packed ? 0 : (int)tokens;
    b->off = offsets;
    return DWCONV_OK;
}

// Row strides may pass 2^31 elements, not the address space.
inline bool ld_ok(long long ld, long long width) { return ld >= width && ld < (1LL << 40); }

// The recurrence and the products address a tile's rows by 32-bit offsets.
inline bool short_ld_ok(long long ld, long long width) { return ld >= width && ld < (1LL << 21); }

inline int check_workspace(const void *ws, long long have, long long need)
{
    if (need > 0 && (!ws || !aligned(ws, 16) || have < need))
        return DWCONV_ERR_WORKSPACE;
    return DWCONV_OK;
}

}  // namespace dwseq
