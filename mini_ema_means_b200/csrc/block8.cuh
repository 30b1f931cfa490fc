// block8.cuh -- host side of the block-scaled FP8 matrices (k_block8.cuh): argument
// checks, launch shapes and the C ABI. Included at the end of emeans.cu.
#pragma once

// CK that also takes the error off the runtime's record, so that no later call finds it.
#define B8_CK(call)                                                                                \
    do {                                                                                           \
        const cudaError_t e_ = (call);                                                             \
        if (e_ != cudaSuccess) {                                                                   \
            cudaGetLastError();                                                                    \
            return fail(EM_E_CUDA, "%s: %s", #call, cudaGetErrorString(e_));                       \
        }                                                                                          \
    } while (0)

namespace {

// Makes a device current for a call and puts the caller's back.
struct DeviceGuard {
    int prev = -1;
    cudaError_t to(int dev) {
        cudaError_t e = cudaGetDevice(&prev);
        if (e != cudaSuccess || prev == dev) {
            prev = -1;
            return e;
        }
        return cudaSetDevice(dev);
    }
    ~DeviceGuard() {
        if (prev >= 0) cudaSetDevice(prev);
    }
};

// The device a pointer's memory is on, or -1 for host memory (and what is no memory).
int device_of(const void* p) {
    cudaPointerAttributes a;
    if (cudaPointerGetAttributes(&a, p) != cudaSuccess) {
        cudaGetLastError();
        return -1;
    }
    return a.type == cudaMemoryTypeDevice || a.type == cudaMemoryTypeManaged ? a.device : -1;
}

// Every given pointer on one device (NULL ones are not asked). *dev: that device.
int same_device(const char* what, const void* const* ptrs, int count, int* dev) {
    *dev = -1;
    for (int i = 0; i < count; ++i) {
        if (!ptrs[i]) continue;
        const int d = device_of(ptrs[i]);
        if (d < 0 && em_device_count() < 1) return fail(EM_E_NODEVICE, "no CUDA device");
        if (d < 0) return fail(EM_E_INVAL, "%s takes device pointers only", what);
        if (*dev >= 0 && d != *dev) return fail(EM_E_INVAL, "%s: memory of two devices (%d and %d)", what, *dev, d);
        *dev = d;
    }
    return EM_OK;
}

constexpr int64_t kB8MaxD = 1ll << 24;
// The kernels count the (row, block) pairs of a call in 31 bits, and look a few past the
// last (2^31 pairs of whole blocks are 270 GB of codes).
constexpr int64_t kB8MaxPairs = (1ll << 31) - (1ll << 16);

int64_t b8_pitch(int64_t d) { return (d + 15) / 16 * 16; }
int64_t b8_blocks(int64_t d) { return (d + b8::kBlock - 1) / b8::kBlock; }
int64_t b8_groups(int64_t d) { return (b8_blocks(d) + 3) / 4; }

int b8_check_shape(int64_t rows, int64_t d) {
    if (rows < 1 || rows >= (1ll << 31) || d < 1 || d > kB8MaxD)
        return fail(EM_E_INVAL, "a block8 matrix needs 1 <= rows < 2^31 and 1 <= d <= 2^24 (rows %lld, d %lld)",
                    (long long)rows, (long long)d);
    return EM_OK;
}

int b8_check(const em_block8_t* m) {
    if (!m) return fail(EM_E_INVAL, "the block8 matrix is NULL");
    CKR(b8_check_shape(m->rows, m->d));
    if (!m->codes || !m->scales || !m->status)
        return fail(EM_E_INVAL, "a block8 matrix needs codes, scales and a status word");
    if (((uintptr_t)m->codes & 15) || ((uintptr_t)m->scales & 15) || ((uintptr_t)m->status & 3) ||
        ((uintptr_t)m->claims & 3))
        return fail(EM_E_INVAL, "block8 codes and scales must be 16-byte aligned, status and claims 4-byte aligned");
    return EM_OK;
}

size_t dtype_size(int dtype) { return dtype == EM_DTYPE_F32 ? 4 : 2; }

int b8_check_dtype(int dtype, const void* p, const char* what) {
    if (dtype != EM_DTYPE_F32 && dtype != EM_DTYPE_BF16 && dtype != EM_DTYPE_F16)
        return fail(EM_E_INVAL, "dtype is 0 (fp32), 1 (bf16) or 2 (fp16), not %d", dtype);
    if ((uintptr_t)p % dtype_size(dtype)) return fail(EM_E_INVAL, "%s is not aligned to its type", what);
    return EM_OK;
}

// Rows [first, first + n) or slots; n within the limits of the row indexes.
int b8_check_rows(const em_block8_t* m, int64_t first, const int64_t* slots, int64_t n) {
    if (n < 0 || n > kB8MaxPairs || n * b8_blocks(m->d) > kB8MaxPairs)
        return fail(EM_E_INVAL, "need 0 <= n and n x ceil(d / 128) <= 2^31 - 2^16 (n = %lld)", (long long)n);
    if (slots) {
        if (first != 0) return fail(EM_E_INVAL, "first must be 0 with slots");
        if ((uintptr_t)slots & 7) return fail(EM_E_INVAL, "slots must be 8-byte aligned");
    } else if (first < 0 || first > m->rows - n) {
        return fail(EM_E_INVAL, "rows [%lld, %lld) are outside the matrix's %lld rows", (long long)first,
                    (long long)(first + n), (long long)m->rows);
    }
    return EM_OK;
}

struct DeviceFacts {
    int sms = 0, clock_khz = 0;
    bool smem_set = false;
};
std::mutex g_b8_mu;
DeviceFacts g_b8_dev[64];

template <class K>
bool b8_smem_attribute(K* kernel, int bytes) {
    return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes) == cudaSuccess;
}

// The current device's SM count and clock; on the first call, its kernels' shared
// memory limits too.
int b8_device(int dev, DeviceFacts* out) {
    if (dev < 0 || dev >= 64) return fail(EM_E_INVAL, "device index out of range");
    std::lock_guard<std::mutex> lock(g_b8_mu);
    DeviceFacts& f = g_b8_dev[dev];
    if (!f.smem_set) {
        int major = 0, minor = 0;
        cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev);
        cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev);
        if (major != 10 || minor != 0) return fail(EM_E_NODEVICE, "this library is built for sm_100a (B200)");
        B8_CK(cudaDeviceGetAttribute(&f.sms, cudaDevAttrMultiProcessorCount, dev));
        B8_CK(cudaDeviceGetAttribute(&f.clock_khz, cudaDevAttrClockRate, dev));
        if (!b8_smem_attribute(b8::k_block8_matmul<128, 4, false>, b8::MmCfg<128, false>::kSmem) ||
            !b8_smem_attribute(b8::k_block8_matmul<128, 2, false>, b8::MmCfg<128, false>::kSmem) ||
            !b8_smem_attribute(b8::k_block8_matmul<128, 4, true>, b8::MmCfg<128, true>::kSmem) ||
            !b8_smem_attribute(b8::k_block8_matmul<128, 2, true>, b8::MmCfg<128, true>::kSmem) ||
            !b8_smem_attribute(b8::k_block8_matmul<32, 4, false>, b8::MmCfg<32, false>::kSmem) ||
            !b8_smem_attribute(b8::k_block8_matmul<32, 2, false>, b8::MmCfg<32, false>::kSmem) ||
            !b8_smem_attribute(b8::k_block8_matmul<32, 4, true>, b8::MmCfg<32, true>::kSmem) ||
            !b8_smem_attribute(b8::k_block8_matmul<32, 2, true>, b8::MmCfg<32, true>::kSmem) ||
            !b8_smem_attribute(b8::k_block8_matmul_pair<4, false>, b8::kSmem2) ||
            !b8_smem_attribute(b8::k_block8_matmul_pair<2, false>, b8::kSmem2) ||
            !b8_smem_attribute(b8::k_block8_matmul_pair<4, true>, b8::kSmem2Ast) ||
            !b8_smem_attribute(b8::k_block8_matmul_pair<2, true>, b8::kSmem2Ast)) {
            cudaGetLastError();
            return fail(EM_E_CUDA, "cudaFuncSetAttribute failed");
        }
        f.smem_set = true;
    }
    *out = f;
    return EM_OK;
}

// Blocks per SM at most: many more than fit, so that the last ones even out (65,536 x
// 768 bf16 written in 23.7 us, with 8 per SM in 27.5; read back to fp32 39.0 and 42.7).
constexpr int kB8PerSm = 64;

int b8_pair_grid(int64_t n, int64_t nb, int sms) {
    return grid_for((n * nb + b8::kPairsPerWarp - 1) / b8::kPairsPerWarp * 32, 256, sms, kB8PerSm);
}

template <class T>
int b8_write(bool cols, const void* X_, int64_t n, int64_t ldx, const int64_t* slots, int64_t first, const int* claims,
             const em_block8_t* m, int sms, cudaStream_t st) {
    const T* X = static_cast<const T*>(X_);
    uint8_t* codes = static_cast<uint8_t*>(m->codes);
    uint8_t* scales = static_cast<uint8_t*>(m->scales);
    const int64_t nb = b8_blocks(m->d);
    const int d = (int)m->d, pitch = (int)b8_pitch(m->d);
    if (!cols) {
        if (d % 16 == 0 && (uintptr_t)X % 32 == 0 && ldx * sizeof(T) % 32 == 0) {
            B8_CK(launch_k(true, slots ? b8::k_block8_write_wide<T, true> : b8::k_block8_write_wide<T, false>,
                        dim3(b8_pair_grid(n, nb, sms)), dim3(256), 0, st, X, (int)n, d, ldx, slots, (int)first, claims,
                        codes, scales, m->rows, b8::FastDiv((uint32_t)nb), m->status));
            return EM_OK;
        }
        const int width = b8::vector_width<T>(X, ldx);
        const bool fast = width * sizeof(T) == 16 && d % 8 == 0;
        auto* kernel = slots ? (fast ? b8::k_block8_write<T, true, true> : b8::k_block8_write<T, true, false>)
                             : (fast ? b8::k_block8_write<T, false, true> : b8::k_block8_write<T, false, false>);
        B8_CK(launch_k(true, kernel, dim3(b8_pair_grid(n, nb, sms)), dim3(256), 0, st, X, (int)n, d, ldx, width, slots,
                    (int)first, claims, codes, scales, m->rows, pitch, b8::FastDiv((uint32_t)nb), m->status));
        return EM_OK;
    }
    const int64_t row_tiles = (n + b8::ColTile<T>::kRows - 1) / b8::ColTile<T>::kRows;
    const int grid = (int)std::min<int64_t>(row_tiles * nb, (int64_t)sms * kB8PerSm);
    B8_CK(launch_k(true, b8::k_block8_write_cols<T>, dim3(grid), dim3(256), 0, st, X, (int)n, d, ldx,
                b8::vector_width<T>(X, ldx), slots, first, claims, codes, scales, m->rows, pitch, b8::FastDiv((uint32_t)row_tiles), m->status));
    return EM_OK;
}

template <class T>
int b8_read_as(const em_block8_t* m, int64_t first, const int64_t* slots, int64_t n, void* out, int64_t ldo,
               int64_t columns, int sms, cudaStream_t st) {
    const int64_t nb = b8_blocks(m->d);
    const dim3 grid(b8_pair_grid(n, nb, sms));
    const auto codes = static_cast<const uint8_t*>(m->codes), scales = static_cast<const uint8_t*>(m->scales);
    T* rows_out = static_cast<T*>(out);
    if (columns == m->d && m->d % 16 == 0 && (uintptr_t)out % 32 == 0 && ldo * sizeof(T) % 32 == 0) {
        B8_CK(launch_k(true, slots ? b8::k_block8_read_wide<T, true> : b8::k_block8_read_wide<T, false>, grid, dim3(256), 0,
                    st, codes, scales, m->rows, (int)m->d, slots, (int)first, (int)n, rows_out, ldo,
                    b8::FastDiv((uint32_t)nb), m->status));
        return EM_OK;
    }
    const int width = b8::vector_width<T>(out, ldo);
    if (width == 1) {
        B8_CK(launch_k(true, slots ? b8::k_block8_read_any<T, true> : b8::k_block8_read_any<T, false>, grid, dim3(256), 0,
                       st, codes, scales, m->rows, (int)b8_pitch(m->d), (int)m->d, slots, (int)first, (int)n, rows_out,
                       ldo, (int)columns, b8::FastDiv((uint32_t)nb), m->status));
        return EM_OK;
    }
    B8_CK(launch_k(true, slots ? b8::k_block8_read<T, true> : b8::k_block8_read<T, false>, grid, dim3(256), 0, st, codes,
                   scales, m->rows, (int)b8_pitch(m->d), (int)m->d, slots, (int)first, (int)n, rows_out, ldo, (int)columns,
                   width, b8::FastDiv((uint32_t)nb), m->status));
    return EM_OK;
}

// Reads rows with no checks but the kernel's own (`columns` values per row, zeros past d).
int b8_read(const em_block8_t* m, int64_t first, const int64_t* slots, int64_t n, void* out, int dtype, int64_t ldo,
            int64_t columns, int sms, cudaStream_t st) {
    switch (dtype) {
        case EM_DTYPE_F32: return b8_read_as<float>(m, first, slots, n, out, ldo, columns, sms, st);
        case EM_DTYPE_BF16: return b8_read_as<__nv_bfloat16>(m, first, slots, n, out, ldo, columns, sms, st);
        default: return b8_read_as<__half>(m, first, slots, n, out, ldo, columns, sms, st);
    }
}

}  // namespace

// Whether the rows [0, n) of a block8 matrix can be a model's data.
static int check_block8(const em_model* m, const em_block8_t* x, int64_t n) {
    CKR(b8_check(x));
    if (x->d != m->d || n > x->rows)
        return fail(EM_E_INVAL, "the block8 matrix is %lld x %lld: the model needs %lld rows of %lld values",
                    (long long)x->rows, (long long)x->d, (long long)n, (long long)m->d);
    CKR(b8_check_rows(x, 0, nullptr, n));
    const void* ptrs[] = {x->codes, x->scales, x->status};
    int dev;
    CKR(same_device("a block8 input", ptrs, 3, &dev));
    if (dev != m->dev) return fail(EM_E_INVAL, "the block8 matrix is on device %d, the model on %d", dev, m->dev);
    return EM_OK;
}

// The rows [0, n) of a block8 matrix as a model's bf16 data (pitch m->ld, zeros past d).
static int read_block8(em_model* m, const em_block8_t* x, int64_t n, __nv_bfloat16* out) {
    return b8_read(x, 0, nullptr, n, out, EM_DTYPE_BF16, m->ld, m->ld, m->sms, m->stream);
}

namespace {

// Tensor map over a matrix's exponents: one row of 512 bytes for each 128 rows x 4 blocks.
int b8_scale_map(CUtensorMap* tm, const em_block8_t* m) {
    EncodeTiledFn fn = encode_fn();
    if (!fn) return fail(EM_E_CUDA, "cuTensorMapEncodeTiled is not available");
    cuuint64_t dims[2] = {128, (cuuint64_t)((m->rows + 127) / 128 * b8_groups(m->d))};
    cuuint64_t strides[1] = {b8::kAtomBytes};
    cuuint32_t box[2] = {128, 1}, estr[2] = {1, 1};
    CUresult r = fn(tm, CU_TENSOR_MAP_DATA_TYPE_UINT32, 2, m->scales, dims, strides, box, estr,
                    CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                    CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    if (r != CUDA_SUCCESS) return fail(EM_E_CUDA, "cuTensorMapEncodeTiled (exponents) failed (%d)", (int)r);
    return EM_OK;
}

// Tensor map over the result for the pair kernel's stores: boxes of 32 rows x 128 bytes.
int b8_out_map(CUtensorMap* tm, const b8::MmArgs& p, size_t esz) {
    EncodeTiledFn fn = encode_fn();
    if (!fn) return fail(EM_E_CUDA, "cuTensorMapEncodeTiled is not available");
    cuuint64_t dims[2] = {(cuuint64_t)p.n_rows, (cuuint64_t)p.m_rows};
    cuuint64_t strides[1] = {(cuuint64_t)p.ldo * esz};
    cuuint32_t box[2] = {(cuuint32_t)(128 / esz), 32}, estr[2] = {1, 1};
    CUresult r = fn(tm, esz == 4 ? CU_TENSOR_MAP_DATA_TYPE_UINT32 : CU_TENSOR_MAP_DATA_TYPE_UINT16, 2, p.out, dims, strides,
                    box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                    CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    if (r != CUDA_SUCCESS) return fail(EM_E_CUDA, "cuTensorMapEncodeTiled (result) failed (%d)", (int)r);
    return EM_OK;
}

template <int BN, bool SWAP>
int b8_launch_single(const CUtensorMap& tmA, const CUtensorMap& tmB, const CUtensorMap& tmSA, const CUtensorMap& tmSB,
                     b8::MmArgs p, size_t esz, int sms, cudaStream_t st) {
    const int64_t tiles = (int64_t)p.m_tiles * p.n_tiles;
    // Rows of several spans, where a CTA for each span of each tile still fits the SMs at
    // once: a cluster per tile. It pays from 3 spans on with 128 x 32 tiles (16 x 512: d =
    // 2,048 6.1 us and 6.4 without, 8,192 8.0 and 18.1), from 4 with the larger ones, whose
    // results take longer to meet (200 x 300: 2,048 10.1 and 9.5, 4,096 12.4 and 13.6).
    const int64_t spans = (p.nkb + b8::kSpan - 1) / b8::kSpan;
    p.split = spans >= (BN == 32 ? 3 : 4) && spans <= 8 && tiles * spans <= sms ? (int)spans : 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(p.split > 1 ? tiles * spans : std::min<int64_t>(tiles, sms)));
    cfg.blockDim = dim3(b8::kMmThreads);
    cfg.dynamicSmemBytes = b8::MmCfg<BN, SWAP>::kSmem;
    cfg.stream = st;
    cudaLaunchAttribute attr[2] = {};
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)p.split;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = p.split > 1 ? 2 : 1;
    B8_CK(cudaLaunchKernelEx(&cfg, esz == 4 ? b8::k_block8_matmul<BN, 4, SWAP> : b8::k_block8_matmul<BN, 2, SWAP>, tmA, tmB,
                             tmSA, tmSB, p));
    return EM_OK;
}

// A product with the rows of `a` on the tiles' M side; `swap`: they are the output's columns.
int b8_launch_matmul(const em_block8_t* a, int64_t na, const em_block8_t* b, int64_t nb, bool swap, b8::MmArgs p,
                     size_t esz, int sms, cudaStream_t st) {
    // Pairs of CTAs with 256 x 192 tiles, or single ones with 128 x 128: the one whose
    // longest CTA is shorter (per block 384 cycles a pair tile, about 400 a single one,
    // which L2 feeds).
    const int64_t t1 = ((na + 127) / 128) * ((nb + 127) / 128);
    const int64_t t2 = ((na + 255) / 256) * ((nb + b8::kPairN - 1) / b8::kPairN);
    const int64_t pairs = std::max(sms / 2, 1);
    const bool narrow = nb <= 32;
    const bool pair = !swap && !narrow && t1 > sms && (t2 + pairs - 1) / pairs * 384 <= (t1 + sms - 1) / sms * 400;
    const int box_b = pair ? b8::kPairN / 2 : narrow ? 32 : 128;
    CUtensorMap tmA, tmB, tmSA, tmSB;
    CKR(make_tmap8(&tmA, a->codes, a->rows, (int)a->d, (int)b8_pitch(a->d), 128));
    CKR(make_tmap8(&tmB, b->codes, b->rows, (int)b->d, (int)b8_pitch(b->d), box_b));
    CKR(b8_scale_map(&tmSA, a));
    CKR(b8_scale_map(&tmSB, b));
    p.m_rows = na;
    p.n_rows = nb;
    p.nkb = (int)b8_blocks(a->d);
    if (pair) {
        p.m_tiles = (int)((na + 255) / 256);
        p.n_tiles = (int)((nb + b8::kPairN - 1) / b8::kPairN);
        // (strides of a tensor map end below 2^40 bytes)
        if (p.ldo * (int64_t)esz >= (1ll << 40)) p.vec_ok = 0;
        CUtensorMap tmOut = tmA;  // not used where the result's rows are not aligned
        if (p.vec_ok) CKR(b8_out_map(&tmOut, p, esz));
        // A stationary where the MMAs of a tile outlast its stores (65,536 x 4,096: bf16
        // results at d = 384 131 us, 136 without, at 768 204 and 217; fp32 at 768 251 and
        // 264). Below that the stores count, and consecutive tiles on one pair spread the
        // pairs' stores over memory (fp32 at d = 384 225 us, 191 without; bf16 at 256 123
        // and 116).
        const bool ast = p.nkb <= b8::kAstBlocks && 2 * p.nkb >= 3 * (int)esz;
        auto* kernel = esz == 4 ? (ast ? b8::k_block8_matmul_pair<4, true> : b8::k_block8_matmul_pair<4, false>)
                                : (ast ? b8::k_block8_matmul_pair<2, true> : b8::k_block8_matmul_pair<2, false>);
        B8_CK(launch_k(true, kernel, dim3((unsigned)(2 * std::min(t2, pairs))), dim3(b8::kPairThreads),
                    ast ? b8::kSmem2Ast : b8::kSmem2, st, tmA, tmB, tmSA, tmSB, tmOut, p));
        return EM_OK;
    }
    p.m_tiles = (int)((na + 127) / 128);
    p.n_tiles = (int)((nb + box_b - 1) / box_b);
    if (narrow)
        return swap ? b8_launch_single<32, true>(tmA, tmB, tmSA, tmSB, p, esz, sms, st)
                    : b8_launch_single<32, false>(tmA, tmB, tmSA, tmSB, p, esz, sms, st);
    if (swap) return b8_launch_single<128, true>(tmA, tmB, tmSA, tmSB, p, esz, sms, st);
    return b8_launch_single<128, false>(tmA, tmB, tmSA, tmSB, p, esz, sms, st);
}

}  // namespace

extern "C" {

int em_block8_layout(int64_t rows, int64_t d, int64_t* pitch, int64_t* code_bytes, int64_t* scale_bytes) {
    CKR(b8_check_shape(rows, d));
    if (pitch) *pitch = b8_pitch(d);
    if (code_bytes) *code_bytes = rows * b8_pitch(d);
    if (scale_bytes) *scale_bytes = (rows + 127) / 128 * b8_groups(d) * b8::kAtomBytes;
    return EM_OK;
}

int em_block8_write(const em_block8_t* m, const void* X, int dtype, int64_t n, int64_t row_stride, int64_t col_stride,
                    int64_t first, const int64_t* slots, void* stream) {
    CKR(b8_check(m));
    CKR(b8_check_dtype(dtype, X, "X"));
    CKR(b8_check_rows(m, first, slots, n));
    if (row_stride < 0 || col_stride < 0 || (row_stride != 1 && col_stride != 1))
        return fail(EM_E_INVAL, "one of row_stride and col_stride must be 1, and neither negative");
    if (n == 0) return EM_OK;
    if (!X) return fail(EM_E_INVAL, "X is NULL");
    if (slots && n > b8::kScanRows && !m->claims)
        return fail(EM_E_INVAL, "writing more than %d rows by slots needs the matrix's claims array", b8::kScanRows);
    const void* ptrs[] = {m->codes, m->scales, m->claims, m->status, X, slots};
    int dev;
    CKR(same_device("em_block8_write", ptrs, 6, &dev));
    DeviceGuard guard;
    B8_CK(guard.to(dev));
    DeviceFacts f;
    CKR(b8_device(dev, &f));
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const int* claims = nullptr;
    if (slots && n > b8::kScanRows) {
        B8_CK(launch_k(true, b8::k_block8_claim, dim3(grid_for(n, 256, f.sms)), dim3(256), 0, st, slots, n, m->rows,
                    m->claims));
        claims = m->claims;
    }
    const bool cols = col_stride != 1;
    const int64_t ldx = cols ? col_stride : row_stride;
    switch (dtype) {
        case EM_DTYPE_F32: return b8_write<float>(cols, X, n, ldx, slots, first, claims, m, f.sms, st);
        case EM_DTYPE_BF16: return b8_write<__nv_bfloat16>(cols, X, n, ldx, slots, first, claims, m, f.sms, st);
        default: return b8_write<__half>(cols, X, n, ldx, slots, first, claims, m, f.sms, st);
    }
}

int em_block8_read(const em_block8_t* m, int64_t first, const int64_t* slots, int64_t n, void* out, int dtype,
                   int64_t row_stride, void* stream) {
    CKR(b8_check(m));
    CKR(b8_check_dtype(dtype, out, "out"));
    CKR(b8_check_rows(m, first, slots, n));
    if (row_stride < m->d) return fail(EM_E_INVAL, "row_stride is below d");
    if (n == 0) return EM_OK;
    if (!out) return fail(EM_E_INVAL, "out is NULL");
    const void* ptrs[] = {m->codes, m->scales, m->status, out, slots};
    int dev;
    CKR(same_device("em_block8_read", ptrs, 5, &dev));
    DeviceGuard guard;
    B8_CK(guard.to(dev));
    DeviceFacts f;
    CKR(b8_device(dev, &f));
    return b8_read(m, first, slots, n, out, dtype, row_stride, m->d, f.sms, static_cast<cudaStream_t>(stream));
}

int em_block8_matmul(const em_block8_t* a, int64_t na, const em_block8_t* b, int64_t nb, void* out, int dtype,
                     int64_t row_stride, void* stream) {
    CKR(b8_check(a));
    CKR(b8_check(b));
    CKR(b8_check_dtype(dtype, out, "out"));
    if (a->d != b->d)
        return fail(EM_E_INVAL, "the matrices have rows of %lld and %lld values", (long long)a->d, (long long)b->d);
    if (na < 0 || na > a->rows || nb < 0 || nb > b->rows)
        return fail(EM_E_INVAL, "na and nb must be within the matrices' rows");
    if (row_stride < nb) return fail(EM_E_INVAL, "row_stride is below nb");
    if (na == 0 || nb == 0) return EM_OK;
    if (!out) return fail(EM_E_INVAL, "out is NULL");
    const void* ptrs[] = {a->codes, a->scales, a->status, b->codes, b->scales, out};
    int dev;
    CKR(same_device("em_block8_matmul", ptrs, 6, &dev));
    DeviceGuard guard;
    B8_CK(guard.to(dev));
    DeviceFacts f;
    CKR(b8_device(dev, &f));
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    b8::MmArgs p = {};
    p.out = out;
    p.ldo = row_stride;
    p.bf16 = dtype == EM_DTYPE_BF16;
    p.wait_limit = 2000ll * f.clock_khz;
    p.status = a->status;
    const size_t esz = dtype_size(dtype);
    p.vec_ok = (uintptr_t)out % 16 == 0 && row_stride * esz % 16 == 0;
    // few output rows: the rows of b take the tiles' 128 lanes
    if (na <= 128 && nb > na) return b8_launch_matmul(b, nb, a, na, true, p, esz, f.sms, st);
    return b8_launch_matmul(a, na, b, nb, false, p, esz, f.sms, st);
}

int em_block8_check(const em_block8_t* m, void* stream) {
    CKR(b8_check(m));
    const void* ptrs[] = {m->status};
    int dev;
    CKR(same_device("em_block8_check", ptrs, 1, &dev));
    DeviceGuard guard;
    B8_CK(guard.to(dev));
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    cudaStreamCaptureStatus capturing = cudaStreamCaptureStatusNone;
    B8_CK(cudaStreamIsCapturing(st, &capturing));
    if (capturing != cudaStreamCaptureStatusNone)
        return fail(EM_E_STATE, "em_block8_check waits for the stream: not while it is captured");
    int32_t h = 0;
    B8_CK(cudaMemcpyAsync(&h, m->status, sizeof(h), cudaMemcpyDeviceToHost, st));
    B8_CK(cudaStreamSynchronize(st));
    if (h != 0) {
        B8_CK(cudaMemsetAsync(m->status, 0, sizeof(h), st));
        B8_CK(cudaStreamSynchronize(st));
        return fail(h, h == EM_E_TIMEOUT ? "a device-side wait exceeded its limit"
                                         : "a slot is outside the matrix (device error %d)",
                    (int)h);
    }
    return EM_OK;
}

}  // extern "C"
