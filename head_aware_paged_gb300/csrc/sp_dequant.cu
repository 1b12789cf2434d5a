// sp_dequant.cu -- 4-bit history pages -> bf16 rows in the workspace, ahead of
// a prefill over them.  A unit's slots follow one another there, so a tile of
// k_prefill is one 128-row box whatever the page size.
//
// Every query tile of a chunk reads the same history, so its codes are turned
// into bf16(code * scale * channel scale) once per call instead of once per
// work item: a converter inside k_prefill (two warps next to eight softmax
// warps) took about 8,000 cycles for the K and V of a tile whose products take
// 2,048, and a fourth warpgroup of converters cost the softmax its registers
// (2,048 rows after 16,384: 188 us that way, 121 us this way, 127 us on bf16
// pages of 64).  Bound by memory: 144 bytes read and 512 written a key, most of which
// stay in L2 for the kernel that follows; a short history is a launch and one
// chain of loads, so a thread issues all of a page's at once (with them in a
// loop over rows, every head GLOBAL: 505 instead of 498 us for the call).
//
// code * scale has 6 significant bits, exact in bf16; a channel scale that is not
// a power of two makes it 2^-8 relative, the step of the rows that the chunk
// itself brings.
#include "sp_device.cuh"
#include "sp_internal.h"

namespace sp {

namespace {

// One block per (unit, page) of the call, grid-strided.  A thread converts one
// block of 16 dimensions of a row, NI times: rows (tid / 8) + 32 i of the
// page's K rows and then its V rows, 2 P = 32 NI in all, every load issued
// before the first conversion; eight neighbours write a row's 256 bytes.
template <int NI>
__global__ void __launch_bounds__(256) k_dequant4(const __grid_constant__ DequantParams p) {
    const Geo& g = p.geo;
    constexpr int P = 16 * NI;
    const int D = g.d;
    const int total = p.page_off[p.n_units];
    const int c = threadIdx.x & 7;                   // this thread's block of a row
    for (int blk = blockIdx.x; blk < total; blk += gridDim.x) {
        int a = 0, z = p.n_units - 1;                // unit with page_off[u] <= blk < page_off[u + 1]
        while (a < z) {
            const int mid = (a + z + 1) >> 1;
            if (p.page_off[mid] <= blk) a = mid; else z = mid - 1;
        }
        const int u = p.unit0 + a, pg = blk - p.page_off[a];
        const int b = u / g.hkv, h = u - b * g.hkv;
        const int64_t row = g.unit_row(p.seq[b], p.layer, h);
        int32_t phys = p.meta.ptab[row * g.max_pages_unit + pg];
        if (phys < 0 || phys >= g.num_pages) {       // the same for the whole block
            if (threadIdx.x == 0) atomicOr(p.meta.status, kStatusBadPage);
            phys = 0;                                // convert something harmless
        }
        if (threadIdx.x == 0 && pg == 0) p.row0[u] = blk * P;
        uint2 code[NI];
        uint32_t scale[NI];
        #pragma unroll
        for (int i = 0; i < NI; ++i) {
            const int at = (threadIdx.x >> 3) + 32 * i, r = at & (P - 1), s = r & 15;
            const bool v = at >= P;
            const uint8_t* grp = (v ? p.vpool : p.kpool) + fp4_group_off(phys, r, P);
            code[i] = __ldg(reinterpret_cast<const uint2*>(grp + (v ? fp4_v_code(s, c) : fp4_k_code(s, c))));
            scale[i] = __ldg(grp + (v ? fp4_v_scale(s, c) : fp4_k_scale(s, c)));
        }
        #pragma unroll
        for (int i = 0; i < NI; ++i) {
            const int at = (threadIdx.x >> 3) + 32 * i, r = at & (P - 1);
            const bool v = at >= P;
            float x[16];
            fp4_value16(code[i], scale[i], x);
            if (p.scaled) {
                const float* cs = (v ? p.meta.vscale : p.meta.kscale) + ((int64_t)p.layer * g.hkv + h) * D + c * 16;
                #pragma unroll
                for (int e = 0; e < 16; e += 4) {
                    const float4 f = __ldg(reinterpret_cast<const float4*>(cs + e));
                    x[e] *= f.x; x[e + 1] *= f.y; x[e + 2] *= f.z; x[e + 3] *= f.w;
                }
            }
            uint32_t o[8];
            #pragma unroll
            for (int e = 0; e < 8; ++e) o[e] = pack_bf16(x[2 * e], x[2 * e + 1]);
            st_global_v8((v ? p.v : p.k) + ((int64_t)blk * P + r) * D + c * 16,
                         o[0], o[1], o[2], o[3], o[4], o[5], o[6], o[7]);
        }
    }
}

static_assert(sizeof(DequantParams) <= 32764, "dequantisation parameters exceed the kernel parameter space");

}  // namespace

cudaError_t launch_dequant4(const sp_cache* c, const DequantParams& p, cudaStream_t s) {
    const int total = p.page_off[p.n_units];
    if (total <= 0) return cudaSuccess;
    const int grid = total < 16 * c->num_sms ? total : 16 * c->num_sms;
    switch (c->geo.page) {
        case 16: k_dequant4<1><<<grid, 256, 0, s>>>(p); break;
        case 32: k_dequant4<2><<<grid, 256, 0, s>>>(p); break;
        case 64: k_dequant4<4><<<grid, 256, 0, s>>>(p); break;
        case 128: k_dequant4<8><<<grid, 256, 0, s>>>(p); break;
        default: return cudaErrorInvalidValue;
    }
    return cudaGetLastError();
}

}  // namespace sp
