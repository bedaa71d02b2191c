// Argument checks shared by the entry points of the layer operators: alignment, workspaces, and outputs that share bytes
// with inputs or with one another.
#pragma once

#include <initializer_list>

#include "api_common.h"
#include "gla.h"

namespace gla {

inline bool any_misaligned(std::initializer_list<const void *> ps)
{
    for (const void *p : ps)
        if (misaligned(p))
            return true;
    return false;
}

inline int check_workspace(const void *workspace, size_t have, size_t need)
{
    if (!workspace || have < need)
        return GLA_ERR_WORKSPACE;
    return reinterpret_cast<uintptr_t>(workspace) % kAlign ? GLA_ERR_ALIGNMENT : GLA_OK;
}

// The bytes of `rows` rows of `width` bytes that start `pitch` bytes apart.
struct Rows {
    uintptr_t lo, hi;
    size_t pitch, width;
};

inline Rows rows_of(const void *p, size_t rows, size_t width, size_t pitch)
{
    const uintptr_t a = reinterpret_cast<uintptr_t>(p);
    return {a, p && rows && width ? a + (rows - 1) * pitch + width : a, pitch, width};
}
inline Rows flat(const void *p, size_t bytes) { return rows_of(p, 1, bytes, bytes); }

// Whether the two share bytes.  Column ranges of one row-strided tensor (equal pitches) interleave without sharing.
inline bool share(const Rows &a, const Rows &b)
{
    if (!overlap({a.lo, a.hi}, {b.lo, b.hi}))
        return false;
    if (a.pitch != b.pitch)
        return true;
    const uintptr_t lo = a.lo < b.lo ? a.lo : b.lo, hi = a.lo < b.lo ? b.lo : a.lo;
    const size_t at = (hi - lo) % a.pitch;
    const size_t first = a.lo < b.lo ? a.width : b.width, second = a.lo < b.lo ? b.width : a.width;
    return at < first || at + second > a.pitch;
}

template <size_t NO, size_t NI>
bool outputs_clash(const Rows (&out)[NO], const Rows (&in)[NI])
{
    for (size_t i = 0; i < NO; ++i) {
        for (size_t j = 0; j < NI; ++j)
            if (share(out[i], in[j]))
                return true;
        for (size_t j = i + 1; j < NO; ++j)
            if (share(out[i], out[j]))
                return true;
    }
    return false;
}

}  // namespace gla
