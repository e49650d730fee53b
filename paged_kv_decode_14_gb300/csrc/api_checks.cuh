// Argument checks that entry points share.
#pragma once

#include "common.cuh"

namespace pkv {

pkv_status check_cache(const pkv_cache* c);

inline bool aligned16(const void* p) { return ((uintptr_t)p & 15) == 0; }

// Rows the kernels may touch in 16-byte pieces; out: no two of them share memory (all heads of a token lie
// between two tokens' starts, or all tokens of a head between two heads').
inline bool rows_ok(const pkv_rows* r, int64_t tokens, int elem_bytes, int head_dim, bool out) {
    if (!r || !r->data || r->num_heads < 1 || !aligned16(r->data)) return false;
    if (tokens > 1 && (r->token_stride * elem_bytes) % 16) return false;
    if (r->num_heads > 1 && (r->head_stride * elem_bytes) % 16) return false;
    if (!out || (tokens <= 1 && r->num_heads == 1)) return true;
    const __int128 ts = tokens > 1 ? r->token_stride : 0, hs = r->num_heads > 1 ? r->head_stride : 0;
    const __int128 t = ts < 0 ? -ts : ts, h = hs < 0 ? -hs : hs;
    if ((tokens > 1 && t < head_dim) || (r->num_heads > 1 && h < head_dim)) return false;
    return tokens == 1 || r->num_heads == 1 || t >= h * (r->num_heads - 1) + head_dim || h >= t * (tokens - 1) + head_dim;
}

}  // namespace pkv
