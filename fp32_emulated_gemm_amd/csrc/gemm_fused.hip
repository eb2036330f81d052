// gemm_fused.hip -- the BF16x9 kernels with the gated product in the epilogue: it
// runs on a tile's recombined FP32 values before they are stored, which spares a
// pass over the product; or with the adapters' part in the accumulators from the
// start.  6144 x 256 -> 2 x 1024 gated 54 us (119 TFLOP/s effective), 2111 x 1024 x
// 1024 with 8 adapters 58 us with the shrink.
//
// Nine products and the truncating split only.  The plain launchers here are
// those of gemm.hip with the same argument form.
#include "gemm_kernels.hpp"
#include "ops.hpp"

namespace sgemm_emu_dev {

namespace {

using C128 = Cfg8S;

template <class C>
GemmArgs tiled(const GemmArgs &args)
{
    GemmArgs g = args;
    g.tiles_m = (int)((g.M + C::BM - 1) / C::BM);
    g.tiles_n = (int)((g.N + C::BN - 1) / C::BN);
    g.group_m = group_rows(g.tiles_n, g.num_cus);
    return g;
}

// One workgroup per CU, a multiple of 8 so that each stays on one XCD.
dim3 persistent_grid(const GemmArgs &g)
{
    const int64_t units = (int64_t)g.tiles_m * g.tiles_n, slots = g.num_cus > 8 ? g.num_cus & ~7 : 8;
    return dim3((unsigned)(units < slots ? units : slots));
}

// A's rows lie in 16-byte pieces and K is a multiple of 64 (callers copy others
// to padded rows), so only the kernels without element loads or masks are built.
template <int EPI>
hipError_t fused_tile64(const GemmArgs &args, hipStream_t stream)
{
    const GemmArgs g = tiled<Cfg64S>(args);
    hipLaunchKernelGGL((gemm_bf16x9_kernel<Cfg64S, 5, true, B_PLANES_NK, 1, false, EPI>),
                       dim3((unsigned)((int64_t)g.tiles_m * g.tiles_n)), dim3(Cfg64S::NT), 0, stream, g);
    return hipGetLastError();
}

template <int EPI>
hipError_t fused_planes(const GemmArgs &args, hipStream_t stream)
{
    const GemmArgs g = tiled<C128>(args);
    launch_last(gemm_bf16x9_planes_kernel<C128, 5, EPI>, persistent_grid(g), dim3(C128::NT), stream, g);
    return hipGetLastError();
}

template <int EPI>
hipError_t fused_dma(const GemmArgs &args, hipStream_t stream)
{
    const GemmArgs g = tiled<C128>(args);
    const dim3 block(C128::NT);
    if (!aligned(g.A, 16) || g.lda % 4 != 0 || g.ka != g.K) return hipErrorInvalidValue;
#ifdef SGEMM_EMU_SERIAL_LDS
    launch_last(gemm_bf16x9_serial_kernel<C128, 5, true, false, false, EPI>,
                dim3((unsigned)((int64_t)g.tiles_m * g.tiles_n)), block, stream, g);
#else
    if (g.sk_grid == 0) {
        launch_last(gemm_bf16x9_dma_kernel<C128, 5, true, false, false, EPI>, persistent_grid(g), block, stream,
                    g);
    } else if constexpr (EPI == EPI_ADAPTER) {
        // Stream-K's epilogue holds whole partial tiles in registers: with the
        // adapters' start it spilled, 53 us for 6144 x 256 x 1024 against 49 as the
        // product and a pass over C, and 136 against 114 for 3136 x 336 x 3592.
        const hipError_t e = launch_gemm(args, 5, B_PLANES_NK, stream);
        return e != hipSuccess ? e : launch_expand(g.M, g.N, g.epi, g.C, g.ldc, stream);
    } else {
        GemmArgs s = g;
        s.sk_domains = (int)streamk_domains((int64_t)g.tiles_m * g.tiles_n, g.K / (2 * BK), g.sk_grid);
        s.group_m = kStreamkGroupRows;
        launch_last(gemm_bf16x9_streamk_kernel<C128, 5, true, false, false, EPI>, dim3((unsigned)g.sk_grid), block,
                    stream, s);
    }
#endif
    return hipGetLastError();
}

hipError_t plain_tile64(const GemmArgs &g, hipStream_t stream)
{
    return launch_gemm_tile64(g, 5, B_PLANES_NK, stream);
}
hipError_t plain_planes(const GemmArgs &g, hipStream_t stream) { return launch_gemm_planes(g, 5, stream); }
hipError_t plain_dma(const GemmArgs &g, hipStream_t stream) { return launch_gemm(g, 5, B_PLANES_NK, stream); }

}  // namespace

const PlaneLaunchers &plain_launchers()
{
    static const PlaneLaunchers l = {plain_tile64, plain_planes, plain_dma};
    return l;
}

const PlaneLaunchers &gated_launchers()
{
    static const PlaneLaunchers l = {fused_tile64<EPI_GATED>, fused_planes<EPI_GATED>, fused_dma<EPI_GATED>};
    return l;
}

const PlaneLaunchers &adapter_launchers()
{
    static const PlaneLaunchers l = {fused_tile64<EPI_ADAPTER>, fused_planes<EPI_ADAPTER>, fused_dma<EPI_ADAPTER>};
    return l;
}

}  // namespace sgemm_emu_dev
