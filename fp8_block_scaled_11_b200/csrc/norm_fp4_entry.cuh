// norm_fp4_entry.cuh -- C entry points of the RMS norm (norm_kernels.cuh), of the
// microscaled 4-bit quantisation (fp4_quant_kernels.cuh) and of the 4-bit product
// (gemm_fp4_kernel.cuh): argument validation and launches.  Part of fp8bs_lib.cu's
// translation unit, whose helpers it uses.

namespace {

// A launch that may be set up under the tail of the kernel before it (every kernel
// launched so waits for it (griddepcontrol.wait) before it touches memory).
template <typename... P, typename... A>
fp8bs_status launch_early_cluster(void (*k)(P...), dim3 grid, dim3 block, size_t smem, cudaStream_t stream, int cluster,
                                  A... args)
{
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)cluster;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = cluster > 1 ? 2 : 1;
    if (cudaLaunchKernelEx(&cfg, k, static_cast<P>(args)...) != cudaSuccess) return FP8BS_ERR_CUDA;
    return launch_status();
}

template <typename... P, typename... A>
fp8bs_status launch_early(void (*k)(P...), dim3 grid, dim3 block, size_t smem, cudaStream_t stream, A... args)
{
    return launch_early_cluster(k, grid, block, smem, stream, 1, args...);
}

// ---------------------------------------------------------------- RMS norm
// The arguments both forward entry points share.
fp8bs_status check_norm(const NormParams& p, fp8bs_dtype xt, fp8bs_dtype wt)
{
    if (!valid_dtype(xt) || !valid_dtype(wt)) return FP8BS_ERR_UNSUPPORTED;
    if (p.x == nullptr || p.w == nullptr || p.q == nullptr || p.scale == nullptr || p.rows < 1 || p.cols < 1)
        return FP8BS_ERR_INVALID_ARG;
    if (p.rows > INT32_MAX || p.cols > INT32_MAX) return FP8BS_ERR_INVALID_ARG;
    if (!(p.eps >= 0.f)) return FP8BS_ERR_INVALID_ARG;
    // the sum and h come together: without a residual h is x
    if ((p.res == nullptr) != (p.h == nullptr)) return FP8BS_ERR_INVALID_ARG;
    if (p.ldx < p.cols || (p.res != nullptr && (p.ldr < p.cols || p.ldh < p.cols)) ||
        (p.y != nullptr && p.ldy < p.cols))
        return FP8BS_ERR_INVALID_ARG;
    const int64_t e = (int64_t)dtype_size(xt);
    if (!aligned16(p.x) || !aligned16(p.res) || !aligned16(p.h) || !aligned16(p.w) || !aligned16(p.y) ||
        !aligned16(p.q) || !aligned16(p.scale) || (reinterpret_cast<uintptr_t>(p.rstd) & 3))
        return FP8BS_ERR_ALIGNMENT;
    if ((p.ldx * e) % 16 || p.ldq % 16) return FP8BS_ERR_ALIGNMENT;
    if (p.res != nullptr && ((p.ldr * e) % 16 || (p.ldh * e) % 16)) return FP8BS_ERR_ALIGNMENT;
    if (p.y != nullptr && (p.ldy * e) % 16) return FP8BS_ERR_ALIGNMENT;
    return FP8BS_OK;
}

template <typename T, typename W, int BITS>
fp8bs_status launch_norm_rows(DeviceInfo* d, const NormParams& p, cudaStream_t stream)
{
    const int64_t eights = cdiv(p.cols, 8);
    // one eight per thread where few rows would leave the GPU idle otherwise (a
    // row's latency is what counts); else up to four, over which a row's and its
    // groups' own work is spread
    RowShape sh = {(int)round32(eights), 1};
    if (p.rows > 2 * d->num_sms || eights > 1024) sh = row_shape(eights, 512, {4, 2, 1});
    if (sh.vpt == 0) return launch_early(rmsnorm_quant_wide_kernel<T, BITS>, (unsigned)p.rows, 512, 0, stream, p);
    const int ty = (int)std::max<int64_t>(1, std::min<int64_t>({256 / sh.tx, p.rows, sh.tx > 32 ? 8 : 16}));
    const dim3 block((unsigned)sh.tx, (unsigned)(sh.tx == 16 ? (ty + 1) / 2 * 2 : ty));
    const unsigned grid = (unsigned)cdiv(p.rows, block.y);
    const bool full = p.cols == 8 * (int64_t)sh.vpt * sh.tx && p.rows % block.y == 0;
    auto k = sh.vpt == 1 ? rmsnorm_quant_kernel<T, W, BITS, 1, false>
             : sh.vpt == 2 ? rmsnorm_quant_kernel<T, W, BITS, 2, false>
             : !full ? rmsnorm_quant_kernel<T, W, BITS, 4, false> : rmsnorm_quant_kernel<T, W, BITS, 4, true>;
    return launch_early(k, grid, block, 0, stream, p);
}

template <int BITS>
fp8bs_status launch_norm(DeviceInfo* d, const NormParams& p, fp8bs_dtype xt, cudaStream_t stream)
{
    if (xt == FP8BS_BF16)
        return p.w_f32 ? launch_norm_rows<__nv_bfloat16, float, BITS>(d, p, stream)
                       : launch_norm_rows<__nv_bfloat16, __nv_bfloat16, BITS>(d, p, stream);
    return p.w_f32 ? launch_norm_rows<float, float, BITS>(d, p, stream)
                   : launch_norm_rows<float, __nv_bfloat16, BITS>(d, p, stream);
}

template <typename T, int VPT, int THREADS, bool WREG, bool CLUSTER = false>
fp8bs_status launch_back_ring(DeviceInfo* d, const BackPlan& b, const NormBackParams& p, cudaStream_t stream)
{
    auto k = rmsnorm_back_kernel<T, VPT, THREADS, WREG, CLUSTER>;
    constexpr int slot = (sizeof(T) == 4 ? 1 : 0) + (WREG ? 2 : 0) + (VPT >> 1) * 4 + (THREADS > 256 ? 12 : 0) +
                         (CLUSTER ? 24 : 0);
    if (!d->ring_attr_set[slot].load(std::memory_order_acquire)) {
        std::lock_guard<std::mutex> lock(g_mutex);
        if (!d->ring_attr_set[slot].load(std::memory_order_relaxed)) {
            if (cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kRingSmem) != cudaSuccess)
                return FP8BS_ERR_CUDA;
            d->ring_attr_set[slot].store(true, std::memory_order_release);
        }
    }
    RowRing g = {};
    g.src[0] = p.dy;
    g.src[1] = p.h;
    g.src[2] = p.dh;
    g.pitch[0] = p.lddy * (int64_t)sizeof(T);
    g.pitch[1] = p.ldh * (int64_t)sizeof(T);
    g.pitch[2] = p.lddh * (int64_t)sizeof(T);
    g.rows = p.rows;
    g.row_bytes = (uint32_t)(p.cols * sizeof(T));
    g.tx = b.shape.tx;
    g.ty = b.ty;
    g.slots = b.slots;
    g.err = d->err_ptr;
    return launch_early_cluster(k, (unsigned)b.grid, (unsigned)(g.tx * g.ty), b.smem, stream, std::max(1, b.cluster), p, g);
}

template <typename T, bool WREG>
fp8bs_status launch_back_rows(DeviceInfo* d, const BackPlan& b, const NormBackParams& p, cudaStream_t stream)
{
    // one row's threads are over 256 only where the ring leaves room for one CTA
    // (rows of bf16 with four eights a thread, of fp32 with four or two)
    if (b.shape.tx * b.ty > 256) {
        if constexpr (sizeof(T) == 4)
            if (b.shape.vpt == 2) return launch_back_ring<T, 2, 512, WREG>(d, b, p, stream);
        return launch_back_ring<T, 4, 512, WREG>(d, b, p, stream);
    }
    if (b.cluster > 0)
        return b.shape.vpt == 1 ? launch_back_ring<T, 1, 256, WREG, true>(d, b, p, stream)
                                : launch_back_ring<T, 2, 256, WREG, true>(d, b, p, stream);
    if (b.shape.vpt == 1) return launch_back_ring<T, 1, 256, WREG>(d, b, p, stream);
    if (b.shape.vpt == 2) return launch_back_ring<T, 2, 256, WREG>(d, b, p, stream);
    return launch_back_ring<T, 4, 256, WREG>(d, b, p, stream);
}

template <typename T>
fp8bs_status launch_norm_back(DeviceInfo* d, const BackPlan& b, const NormBackParams& p, float* dweight,
                              cudaStream_t stream)
{
    fp8bs_status st;
    if (b.shape.vpt == 0) {
        st = launch_early(rmsnorm_back_dot_kernel<T>, (unsigned)p.rows, 512, 0, stream, p);
        if (st == FP8BS_OK)
            st = launch_early(rmsnorm_back_wide_kernel<T>, dim3((unsigned)cdiv(p.cols, 2048), (unsigned)b.grid), 256, 0,
                              stream, p);
    } else {
        st = (p.w_f32 != 0) == (sizeof(T) == 4) ? launch_back_rows<T, true>(d, b, p, stream)
                                                : launch_back_rows<T, false>(d, b, p, stream);
    }
    if (st != FP8BS_OK || b.cluster > 0) return st;
    return launch_early(rmsnorm_dw_kernel, (unsigned)cdiv(p.cols, 32), 32 * kDwWarps, 0, stream, (const float*)p.part, (int)b.parts,
                        p.cols, dweight);
}

// ---------------------------------------------------------------- 4-bit product
template <int BN>
fp8bs_status launch_fp4(DeviceInfo* d, const CUtensorMap& tW, const CUtensorMap& tT, const Fp4Params& p, int parts,
                        cudaStream_t stream)
{
    auto k = gemm_fp4_kernel<BN>;
    constexpr int slot = BN == 16 ? 0 : BN == 32 ? 1 : BN == 64 ? 2 : 3;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 1;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.blockDim = dim3(kF4Threads, 1, 1);
    cfg.dynamicSmemBytes = Fp4Cfg<BN>::alloc;
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (!d->fp4_attr_set[slot].load(std::memory_order_acquire)) {
        std::lock_guard<std::mutex> lock(g_mutex);
        if (!d->fp4_attr_set[slot].load(std::memory_order_relaxed)) {
            if (cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)Fp4Cfg<BN>::alloc) !=
                cudaSuccess)
                return FP8BS_ERR_CUDA;
            // two CTAs per SM need more than the default share of shared memory
            if (cudaFuncSetAttribute(k, cudaFuncAttributePreferredSharedMemoryCarveout, cudaSharedmemCarveoutMaxShared) !=
                cudaSuccess)
                return FP8BS_ERR_CUDA;
            // clusters of 2, 4 and 8 CTAs that can be resident at once: the GPU's
            // processor groups need not hold a whole number of them.  The query
            // counts one CTA per SM; two fit by Fp4Cfg's limits on registers,
            // shared memory and TMEM (256 CTAs in clusters of four, 24 x 8192 x
            // 5120: 5.5 us, on half as many 6.5).
            for (int i = 1; i <= 3; ++i) {
                attr[0].val.clusterDim.x = 1u << i;
                cfg.gridDim = dim3((unsigned)(d->num_sms >> i << i), 1, 1);
                int nc = 0;
                if (cudaOccupancyMaxActiveClusters(&nc, k, &cfg) != cudaSuccess) return FP8BS_ERR_CUDA;
                d->fp4_clusters[slot][i].store(nc <= d->num_sms >> i ? 2 * nc : nc, std::memory_order_relaxed);
            }
            d->fp4_attr_set[slot].store(true, std::memory_order_release);
        }
    }
    // as many CTAs per tile as planned, or fewer, so that all clusters are resident at once
    int log_parts = 0;
    for (int i = 1; i <= 3; ++i)
        if ((1 << i) <= parts && p.num_units <= d->fp4_clusters[slot][i].load(std::memory_order_relaxed)) log_parts = i;
    attr[0].val.clusterDim.x = 1u << log_parts;
    cfg.gridDim = dim3((unsigned)(p.num_units << log_parts), 1, 1);
    cfg.numAttrs = 2;
    if (cudaLaunchKernelEx(&cfg, k, tW, tT, p) != cudaSuccess) return FP8BS_ERR_CUDA;
    return launch_status();
}

// The pair kernel's attributes, once per device: the pairs that can be resident at
// once, or none where it cannot run as built.
constexpr int kNoPairs = -1;

fp8bs_status fp4_pairs(DeviceInfo* d, int* pairs)
{
    *pairs = d->fp4_pair_clusters.load(std::memory_order_acquire);
    if (*pairs != 0) return FP8BS_OK;
    std::lock_guard<std::mutex> lock(g_mutex);
    *pairs = d->fp4_pair_clusters.load(std::memory_order_relaxed);
    if (*pairs != 0) return FP8BS_OK;
    auto k = gemm_fp4_pair_kernel;
    if (cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)Fp4PairSmem::alloc) != cudaSuccess)
        return FP8BS_ERR_CUDA;
    cudaFuncAttributes fa;
    if (cudaFuncGetAttributes(&fa, k) != cudaSuccess) return FP8BS_ERR_CUDA;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = 2;
    attr.val.clusterDim.y = 1;
    attr.val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(2 * std::max(1, d->num_sms / 2), 1, 1);
    cfg.blockDim = dim3(kF4PairThreads, 1, 1);
    cfg.dynamicSmemBytes = Fp4PairSmem::alloc;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    int nc = 0;
    if (cudaOccupancyMaxActiveClusters(&nc, k, &cfg) != cudaSuccess) return FP8BS_ERR_CUDA;
    // the register hand-over is sized for this exact allocation at launch: with fewer
    // the epilogue's increase could never be granted
    *pairs = fa.numRegs == kF4LaunchRegs && nc > 0 ? nc : kNoPairs;
    d->fp4_pair_clusters.store(*pairs, std::memory_order_release);
    return FP8BS_OK;
}

fp8bs_status launch_fp4_pair(int pairs, const CUtensorMap& tW, const CUtensorMap& tT, const Fp4Params& p,
                             cudaStream_t stream)
{
    // scale tiles as rows of 128-row blocks of 64-bit words: four tiles (2048
    // bytes, the chunks of a step) of one block of B^T, of two blocks of A
    CUtensorMap tSW, tST;
    fp8bs_status st = make_map(&tSW, CU_TENSOR_MAP_DATA_TYPE_INT64, 8, p.sfb, (uint64_t)p.kcs * 64, cdiv(p.N, 128),
                               (uint64_t)p.kcs * kSfTileBytes, 256, 1, CU_TENSOR_MAP_SWIZZLE_NONE);
    if (st == FP8BS_OK)
        st = make_map(&tST, CU_TENSOR_MAP_DATA_TYPE_INT64, 8, p.sfa, (uint64_t)p.kcs * 64, cdiv(p.M, 128),
                      (uint64_t)p.kcs * kSfTileBytes, 256, 2, CU_TENSOR_MAP_SWIZZLE_NONE);
    if (st != FP8BS_OK) return st;
    return launch_early_cluster(gemm_fp4_pair_kernel, (unsigned)(2 * std::min<int64_t>(p.num_units, pairs)),
                                kF4PairThreads, Fp4PairSmem::alloc, stream, 2, tW, tT, tSW, tST, p);
}

// The split-K reduction, as a programmatic dependent of the product.
fp8bs_status launch_reduce(DeviceInfo* d, const float* ws, int splits, int64_t M, int64_t N, int64_t ldw, void* D,
                           int64_t ldd, int out_f32, int vec_out, cudaStream_t stream)
{
    const int64_t chunks = M * ((N + 3) / 4);
    const int grid = (int)std::max<int64_t>(1, std::min<int64_t>(cdiv(chunks, kReduceThreads), (int64_t)d->num_sms * 16));
    return launch_early(splitk_reduce_kernel, grid, kReduceThreads, 0, stream, ws, splits, M, N, ldw, D, ldd, out_f32,
                        vec_out);
}

}  // namespace

extern "C" {

fp8bs_status fp8_rmsnorm_quant_1x128(const void* x, int64_t ldx, const void* residual, int64_t ld_res, fp8bs_dtype xt,
                                     int64_t rows, int64_t cols, const void* weight, fp8bs_dtype wt, float eps,
                                     void* h, int64_t ldh, float* rstd, void* y, int64_t ldy, uint8_t* q, int64_t ldq,
                                     float* scale_inv, int64_t ld_scale, fp8bs_scale_rule rule, cudaStream_t stream)
{
    if (rule != FP8BS_SCALE_RULE_FP32 && rule != FP8BS_SCALE_RULE_POW2) return FP8BS_ERR_UNSUPPORTED;
    const NormParams p = {x, residual, weight, h, rstd, y, q, scale_inv, rows, cols, ldx, ld_res, ldh, ldy, ldq,
                          ld_scale, eps, 1.f / (float)cols, wt == FP8BS_F32, rule == FP8BS_SCALE_RULE_POW2};
    fp8bs_status st = check_norm(p, xt, wt);
    if (st != FP8BS_OK) return st;
    if (ldq < cols || ld_scale < rows) return FP8BS_ERR_INVALID_ARG;
    if (cols % 16 || ld_scale % 4) return FP8BS_ERR_ALIGNMENT;
    DeviceInfo* d = nullptr;
    if ((st = get_device(&d)) != FP8BS_OK) return st;
    return launch_norm<8>(d, p, xt, stream);
}

fp8bs_status fp4_rmsnorm_quant_1x32(const void* x, int64_t ldx, const void* residual, int64_t ld_res, fp8bs_dtype xt,
                                    int64_t rows, int64_t cols, const void* weight, fp8bs_dtype wt, float eps,
                                    void* h, int64_t ldh, float* rstd, void* y, int64_t ldy, uint8_t* q, int64_t ldq,
                                    uint8_t* scale_tiles, cudaStream_t stream)
{
    const NormParams p = {x, residual, weight, h, rstd, y, q, scale_tiles, rows, cols, ldx, ld_res, ldh, ldy, ldq,
                          cdiv(cols, 128), eps, 1.f / (float)cols, wt == FP8BS_F32, 0};
    fp8bs_status st = check_norm(p, xt, wt);
    if (st != FP8BS_OK) return st;
    if (cols % 32) return FP8BS_ERR_ALIGNMENT;
    if (ldq < cols / 2) return FP8BS_ERR_INVALID_ARG;
    DeviceInfo* d = nullptr;
    if ((st = get_device(&d)) != FP8BS_OK) return st;
    return launch_norm<4>(d, p, xt, stream);
}

size_t fp8bs_rmsnorm_backward_workspace_size(int64_t rows, int64_t cols)
{
    if (rows < 1 || cols < 1) return 0;
    // the largest need over the types and over a call with or without dh
    const int sms = num_sms_current();
    size_t n = 0;
    for (int64_t elem = 2; elem <= 4; elem += 2)
        for (int mats = 2; mats <= 3; ++mats) n = std::max(n, plan_back(rows, cols, elem, mats, sms).bytes);
    return n;
}

fp8bs_status fp8bs_rmsnorm_backward(const void* dy, int64_t lddy, const void* h, int64_t ldh, const void* dh,
                                    int64_t lddh, fp8bs_dtype xt, int64_t rows, int64_t cols, const void* weight,
                                    fp8bs_dtype wt, const float* rstd, void* dx, int64_t lddx, float* dweight,
                                    void* workspace, size_t workspace_bytes, cudaStream_t stream)
{
    if (!valid_dtype(xt) || !valid_dtype(wt)) return FP8BS_ERR_UNSUPPORTED;
    if (dy == nullptr || h == nullptr || weight == nullptr || rstd == nullptr || dx == nullptr || dweight == nullptr ||
        rows < 1 || cols < 1 || rows > INT32_MAX || cols > INT32_MAX)
        return FP8BS_ERR_INVALID_ARG;
    if (lddy < cols || ldh < cols || lddx < cols || (dh != nullptr && lddh < cols)) return FP8BS_ERR_INVALID_ARG;
    const int64_t e = (int64_t)dtype_size(xt);
    if (!aligned16(dy) || !aligned16(h) || !aligned16(dh) || !aligned16(weight) || !aligned16(dx) ||
        (reinterpret_cast<uintptr_t>(rstd) & 3) || (reinterpret_cast<uintptr_t>(dweight) & 3))
        return FP8BS_ERR_ALIGNMENT;
    if ((lddy * e) % 16 || (ldh * e) % 16 || (lddx * e) % 16 || (dh != nullptr && (lddh * e) % 16) || cols % 16)
        return FP8BS_ERR_ALIGNMENT;
    DeviceInfo* d = nullptr;
    fp8bs_status st = get_device(&d);
    if (st != FP8BS_OK) return st;
    const BackPlan b = plan_back(rows, cols, e, dh != nullptr ? 3 : 2, d->num_sms);
    if (workspace == nullptr || workspace_bytes < fp8bs_rmsnorm_backward_workspace_size(rows, cols))
        return FP8BS_ERR_WORKSPACE;
    if (!aligned16(workspace)) return FP8BS_ERR_ALIGNMENT;
    const NormBackParams p = {dy, h, dh, weight, rstd, dx, static_cast<float*>(workspace), dweight,
                              reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + b.dot_off), rows, cols, lddy,
                              ldh, lddh, lddx, wt == FP8BS_F32};
    return xt == FP8BS_BF16 ? launch_norm_back<__nv_bfloat16>(d, b, p, dweight, stream)
                            : launch_norm_back<float>(d, b, p, dweight, stream);
}

size_t fp4_scale_tiles_size(int64_t rows, int64_t cols)
{
    if (rows < 1 || cols < 1) return 0;
    return (size_t)cdiv(rows, 128) * (size_t)cdiv(cols, 128) * kSfTileBytes;
}

fp8bs_status fp4_quant_1x32(const void* x, fp8bs_dtype xt, int64_t rows, int64_t cols, int64_t ldx, uint8_t* q,
                            int64_t ldq, uint8_t* scale_tiles, int transpose_out, cudaStream_t stream)
{
    if (!valid_dtype(xt)) return FP8BS_ERR_UNSUPPORTED;
    if (x == nullptr || q == nullptr || scale_tiles == nullptr || rows < 1 || cols < 1 || rows > INT32_MAX ||
        cols > INT32_MAX || (transpose_out != 0 && transpose_out != 1) || ldx < cols)
        return FP8BS_ERR_INVALID_ARG;
    if (!aligned16(x) || !aligned16(q) || !aligned16(scale_tiles) || (ldx * (int64_t)dtype_size(xt)) % 16 || ldq % 16)
        return FP8BS_ERR_ALIGNMENT;
    if (transpose_out ? (rows % 32 || cols % 16) : cols % 32) return FP8BS_ERR_ALIGNMENT;
    if (ldq < (transpose_out ? rows : cols) / 2) return FP8BS_ERR_INVALID_ARG;
    DeviceInfo* d = nullptr;
    fp8bs_status st = get_device(&d);
    if (st != FP8BS_OK) return st;
    const int64_t kcs = cdiv(transpose_out ? rows : cols, 128);
    const int64_t tiles_c = transpose_out ? cdiv(cols, kQ4Cols) : kcs;
    const int64_t tiles = tiles_c * cdiv(rows, transpose_out ? kQ4Rows : 128);
    if (tiles > INT32_MAX) return FP8BS_ERR_INVALID_ARG;
    const bool full = rows % (transpose_out ? kQ4Rows : 128) == 0 && cols % (transpose_out ? kQ4Cols : 128) == 0;
    auto launch = [&](auto kernel, auto* p, auto... more) {
        return launch_early(kernel, (unsigned)tiles, 256, 0, stream, p, rows, cols, ldx, q, ldq, scale_tiles, (int)kcs,
                            more...);
    };
    const int tc = (int)tiles_c;
    auto typed = [&](auto* p) {
        using T = std::remove_const_t<std::remove_pointer_t<decltype(p)>>;
        if (transpose_out)
            return full ? launch(fp4_quant_cols_kernel<T, true>, p, tc) : launch(fp4_quant_cols_kernel<T, false>, p, tc);
        return full ? launch(fp4_quant_rows_kernel<T, true>, p) : launch(fp4_quant_rows_kernel<T, false>, p);
    };
    return xt == FP8BS_BF16 ? typed(static_cast<const __nv_bfloat16*>(x)) : typed(static_cast<const float*>(x));
}

fp8bs_status fp4_dequant_1x32(const uint8_t* q, int64_t ldq, const uint8_t* scale_tiles, int64_t rows, int64_t cols,
                              void* out, fp8bs_dtype ot, int64_t ldo, cudaStream_t stream)
{
    if (!valid_dtype(ot)) return FP8BS_ERR_UNSUPPORTED;
    if (q == nullptr || scale_tiles == nullptr || out == nullptr || rows < 1 || cols < 1 || rows > INT32_MAX ||
        cols > INT32_MAX || ldq < cols / 2 || ldo < cols)
        return FP8BS_ERR_INVALID_ARG;
    if (!aligned16(q) || !aligned16(scale_tiles) || !aligned16(out) || ldq % 16 ||
        (ldo * (int64_t)dtype_size(ot)) % 16 || cols % 32)
        return FP8BS_ERR_ALIGNMENT;
    DeviceInfo* d = nullptr;
    fp8bs_status st = get_device(&d);
    if (st != FP8BS_OK) return st;
    const int64_t tiles = cdiv(rows, 128) * cdiv(cols, 128);
    if (tiles > INT32_MAX) return FP8BS_ERR_INVALID_ARG;
    const unsigned grid = (unsigned)tiles;
    const bool full = rows % 128 == 0 && cols % 128 == 0;
    auto typed = [&](auto* p) {
        using T = std::remove_pointer_t<decltype(p)>;
        return launch_early(full ? fp4_dequant_kernel<T, true> : fp4_dequant_kernel<T, false>, grid, 256, 0, stream, q, ldq,
                            scale_tiles, rows, cols, (int)cdiv(cols, 128), p, ldo);
    };
    return ot == FP8BS_BF16 ? typed(static_cast<__nv_bfloat16*>(out)) : typed(static_cast<float*>(out));
}

size_t fp4_scaled_gemm_workspace_size(int64_t M, int64_t N, int64_t K)
{
    if (M < 1 || N < 1 || K < 1) return 0;
    return plan_fp4(M, N, K, num_sms_current()).ws_bytes;
}

fp8bs_status fp4_scaled_gemm(int64_t M, int64_t N, int64_t K, const uint8_t* A, int64_t lda, const uint8_t* Bt,
                             int64_t ldb, const uint8_t* scale_a, const uint8_t* scale_b, void* D, int64_t ldd,
                             fp8bs_dtype out_dtype, void* workspace, size_t workspace_bytes, cudaStream_t stream)
{
    if (!valid_dtype(out_dtype)) return FP8BS_ERR_UNSUPPORTED;
    if (A == nullptr || Bt == nullptr || scale_a == nullptr || scale_b == nullptr || D == nullptr || M < 1 || N < 1 ||
        K < 32 || M > INT32_MAX || N > INT32_MAX || K > INT32_MAX)
        return FP8BS_ERR_INVALID_ARG;
    if (lda < K / 2 || ldb < K / 2 || ldd < N) return FP8BS_ERR_INVALID_ARG;
    if (K % 32 || lda % 16 || ldb % 16 || !aligned16(A) || !aligned16(Bt) || !aligned16(scale_a) ||
        !aligned16(scale_b) || reinterpret_cast<uintptr_t>(D) % dtype_size(out_dtype))
        return FP8BS_ERR_ALIGNMENT;
    DeviceInfo* d = nullptr;
    fp8bs_status st = get_device(&d);
    if (st != FP8BS_OK) return st;
    Fp4Plan plan = plan_fp4(M, N, K, d->num_sms);
    int pairs = 0;
    if (plan.pair) {
        if ((st = fp4_pairs(d, &pairs)) != FP8BS_OK) return st;
        if (pairs == kNoPairs) {
            plan = plan_fp4(M, N, K, d->num_sms, false);
            plan.splits = 1;                // (the caller was told that no workspace is needed)
        }
    }
    if (plan.splits > 1) {
        if (workspace == nullptr && workspace_bytes == 0) plan.splits = 1;      // split-K disabled by the caller
        else if (workspace == nullptr || workspace_bytes < plan.ws_bytes) return FP8BS_ERR_WORKSPACE;
        else if (!aligned16(workspace)) return FP8BS_ERR_ALIGNMENT;
    }
    CUtensorMap tW, tT;
    if ((st = make_map(&tW, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, Bt, K / 2, N, ldb, 128, kF4Rows,
                       CU_TENSOR_MAP_SWIZZLE_128B)) != FP8BS_OK)
        return st;
    if ((st = make_map(&tT, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, A, K / 2, M, lda, 128,
                       (uint32_t)(plan.pair ? kF4Rows : plan.bn),
                       CU_TENSOR_MAP_SWIZZLE_128B)) != FP8BS_OK)
        return st;
    Fp4Params p;
    p.M = (int32_t)M;
    p.N = (int32_t)N;
    p.K = (int32_t)K;
    p.steps = (int32_t)cdiv(K, plan.pair ? kF4PairStepK : kF4StepK);
    p.kcs = (int32_t)cdiv(K, 128);
    p.tiles_m = plan.tiles_m;
    p.tiles_n = plan.tiles_n;
    p.splits = plan.splits;
    // the weights of a band (as many tiles as fit 32 MB of L2) are read once from
    // memory, A once per band: 16640 x 5120 x 8192 in one band 281 us, in bands of 8
    // of its 20 tiles 291, of 2 313 (sustained)
    p.band = (int32_t)std::min<int64_t>(
        plan.tiles_n, std::max<int64_t>(4, (int64_t)(32 << 20) / ((plan.pair ? kF4Pair : kF4Rows) * cdiv(K, 2))));
    p.num_units = (int64_t)plan.tiles_m * plan.tiles_n * plan.splits;
    p.B = Bt;
    p.ldb = ldb;
    p.sfa = scale_a;
    p.sfb = scale_b;
    p.D = D;
    p.ldd = ldd;
    p.out_f32 = out_dtype == FP8BS_F32;
    p.ws = static_cast<float*>(workspace);
    p.ldw = plan.ldw;
    p.err = d->err_ptr;
    if (plan.pair) return launch_fp4_pair(pairs, tW, tT, p, stream);
    switch (plan.bn) {
    case 16: st = launch_fp4<16>(d, tW, tT, p, plan.parts, stream); break;
    case 32: st = launch_fp4<32>(d, tW, tT, p, plan.parts, stream); break;
    case 64: st = launch_fp4<64>(d, tW, tT, p, plan.parts, stream); break;
    default: st = launch_fp4<128>(d, tW, tT, p, plan.parts, stream); break;
    }
    if (st != FP8BS_OK || plan.splits == 1) return st;
    const int vec_out = aligned16(D) && (ldd * (int64_t)dtype_size(out_dtype)) % 16 == 0;
    return launch_reduce(d, p.ws, plan.splits, M, N, plan.ldw, D, ldd, p.out_f32, vec_out, stream);
}

}  // extern "C"
