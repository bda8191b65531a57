// The paged 4-bit KV cache: its format and what its kernels share.
//
// A row is the D values of one (token, KV head), D = 64 or 128: codes q + 8
// with q in [-8, 7], eight to an int32 word, lowest nibble first (the experts'
// storage), and one bf16 scale s; its values are q * s. Codes are
// [pages][Hkv][page_size][D / 8], scales [pages][Hkv][page_size]. A slot is
// page * page_size + the token's place in the page.
//
// A scale that is not finite stands for a row that held a value that was not:
// it makes NaN of whatever attends that row, and of nothing else.
#pragma once

#include "common.cuh"
#include "kv4_kernels.cuh"

namespace moe {
namespace kv4 {

// What the attention kernels read of the batch, checked on the way in: a value
// outside its range is brought into it and recorded as MOE_ERR_DEVICE.
struct Batch {
    const int32_t *table;    // [B][max_pages] page of each page_size keys
    const int32_t *lens;     // [B] keys, the new tokens' among them
    const int32_t *cu_q;     // [B + 1] first query of each sequence; null: one each
    int B, T, max_pages, shift;   // page_size = 1 << shift
};

struct Seq {
    int q0, nq, len;   // queries [q0, q0 + nq); the last of them sees all len keys
};

__device__ inline Seq seq_of(const Batch &p, int b, Ctrl *ctrl) {
    Seq s;
    int q0 = b, q1 = b + 1;
    if (p.cu_q) {
        q0 = p.cu_q[b];
        q1 = p.cu_q[b + 1];
    }
    s.q0 = min(max(q0, 0), p.T);
    const int e = min(max(q1, s.q0), p.T);
    s.nq = e - s.q0;
    const int len = p.lens[b];
    const long long most = (long long)p.max_pages << p.shift;
    s.len = (int)min((long long)max(len, 0), most);
    if (s.q0 != q0 || e != q1 || s.len != len) set_error(ctrl, MOE_ERR_DEVICE);
    return s;
}

__device__ inline bool finite_bits(uint16_t s) { return (s & 0x7F80u) != 0x7F80u; }

}  // namespace kv4
}  // namespace moe
