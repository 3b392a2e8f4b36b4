// attn_host.h — the host side of the prompt kernels on the emulated device.
#pragma once
#include "emu.h"

#include "kda_attn_tc.cuh"

namespace kda {
namespace {
#ifdef FEW_ROWS  // kernels that are compiled and not run
char smem_raw[1], smem[1];
#else
alignas(1024) uint8_t smem_raw[256 * 1024];  // the kernels' dynamic shared memory
#endif
}

static CUresult encode(CUtensorMap *tm, CUtensorMapDataType, cuuint32_t rank, void *base, const cuuint64_t *dims,
                       const cuuint64_t *, const cuuint32_t *box, const cuuint32_t *, CUtensorMapInterleave,
                       CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill)
{
    tc::Map m{static_cast<const uint16_t *>(base), dims[0], dims[1], rank > 2 ? dims[2] : 0, rank > 3 ? dims[3] : 0};
    for (cuuint32_t i = 0; i < rank; ++i) m.box[i] = box[i];
    std::memcpy(tm, &m, sizeof m);
    return CUDA_SUCCESS;
}
inline PFN_cuTensorMapEncodeTiled_v12000 tensor_map_encoder() { return encode; }
inline DebugKnobs debug_knobs() { return {0, 0}; }
inline void note_launch() {}

// The list as the plan kernel's order allows it: each sequence's last tile first.
inline cudaError_t launch_attn_plan(const AttnProblem &p, int rows, void *workspace, cudaStream_t)
{
    char *ws = static_cast<char *>(workspace);
    AttnTile *t = reinterpret_cast<AttnTile *>(ws + attn_workspace_layout(p, rows, false).tiles);
    const long long most = attn_tiles(p, rows);
    long long n = 0;
    *reinterpret_cast<int *>(ws) = 0;
    for (int s = 0; s < p.N; ++s) {
        const int a = p.cu_seqlens[s], b = p.cu_seqlens[s + 1];
        for (int i = (b - a + rows - 1) / rows - 1; i >= 0; --i) t[n++] = AttnTile{a + i * rows, a, b, 0};
    }
    for (; n < most; ++n) t[n] = AttnTile{0, 0, 0, 0};
    return cudaSuccess;
}
}  // namespace kda

static kda::AttnProblem problem(const void *q, const void *k, const void *v, const int *cu, int N, int B, int T,
                                int Hq, int Hkv, int d, float scale, int ctas, unsigned seed)
{
    emu::ctas = ctas;
    emu::seed = seed;
    emu::shared_memory = reinterpret_cast<uint8_t *>(kda::smem_raw);
    kda::AttnProblem p{};
    p.q = q; p.k = k; p.v = v; p.cu_seqlens = cu;
    p.N = N; p.B = B; p.T = T; p.Hq = Hq; p.Hkv = Hkv; p.d = d;
    p.scale = scale; p.dtype = KDA_DTYPE_BF16; p.tokens = (long long)B * T;
    return p;
}
