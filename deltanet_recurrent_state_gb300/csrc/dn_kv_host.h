// Host-side argument checks that the paged-cache entry points share.
#pragma once

#include <cstddef>
#include <cstdint>

#include "dn.h"
#include "dn_internal.h"

namespace dn {

inline bool kv_dtypes_known(dn_dtype io, dn_dtype cache) {
    return io >= DN_F16 && io <= DN_E4M3 && cache >= DN_F16 && cache <= DN_E4M3;
}
inline bool kv_dtypes_ok(dn_dtype io, dn_dtype cache) {
    return (io == DN_F16 || io == DN_BF16) && (cache == io || cache == DN_E4M3);
}
inline bool kv_shape_ok(int D, int page) {
    return (D == 64 || D == 128 || D == 256) && (page == 16 || page == 32 || page == 64 || page == 128);
}
inline bool kv_pages_ok(int max_pages, int pages, int page) {
    return max_pages >= 0 && pages >= 0 && (long long)max_pages * page <= DN_KV_MAX_TOKENS;
}
inline int page_log2(int page) { return page == 16 ? 4 : page == 32 ? 5 : page == 64 ? 6 : 7; }
// Required pointers and their alignment; an empty pool or table needs none, nor do the lengths of no requests.
inline bool kv_pointers_ok(int B, const void *start, const void *kv_len, const void *table, const void *kc, const void *vc,
                           const void *ke, const void *ve, dn_dtype cache, int pages, int max_pages) {
    if (!start || !aligned(start, 4) || (B > 0 && (!kv_len || !aligned(kv_len, 4)))) return false;
    if (B > 0 && max_pages > 0 && (!table || !aligned(table, 4))) return false;
    if (pages > 0 && (!kc || !vc || !aligned(kc, 16) || !aligned(vc, 16))) return false;
    return cache != DN_E4M3 || pages == 0 || (ke && ve && aligned(ke, 16) && aligned(ve, 16));
}

}  // namespace dn
