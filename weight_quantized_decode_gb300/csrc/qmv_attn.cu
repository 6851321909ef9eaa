// qmv_attn.cu -- attention over the paged cache, host side: which kernel a call
// runs on, the tensor maps of the cache, the workspace.
#include <cuda.h>

#include <mutex>

#include "qmv_attn.cuh"

namespace qmv {

namespace {

using EncodeTiledFn = CUresult (*)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *,
                                   const cuuint64_t *, const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave,
                                   CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiledFn encode_fn()
{
    static EncodeTiledFn fn = nullptr;
    static std::once_flag once;
    std::call_once(once, [] {
        void *ptr = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &ptr, 12000, cudaEnableDefault, &q) ==
                cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<EncodeTiledFn>(ptr);
    });
    return fn;
}

}  // namespace

bool encode_rows(CUtensorMap *map, const AttnParams &p, const void *base, int D, int kind, int rows)
{
    EncodeTiledFn enc = encode_fn();
    if (!enc) return false;
    const int esz = kind == kKvF16 ? 2 : 1;
    const int inner = D * esz < 128 ? D : 128 / esz;
    const cuuint64_t dims[3] = {static_cast<cuuint64_t>(D), static_cast<cuuint64_t>(p.Hkv) << p.page_shift,
                                static_cast<cuuint64_t>(p.n_pages)};
    const cuuint64_t strides[2] = {static_cast<cuuint64_t>(D * esz), static_cast<cuuint64_t>(p.page_stride) * esz};
    const cuuint32_t box[3] = {static_cast<cuuint32_t>(inner), static_cast<cuuint32_t>(rows), 1};
    const cuuint32_t estr[3] = {1, 1, 1};
    return enc(map, kind == kKvF16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_UINT8, 3,
               const_cast<void *>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
               inner * esz == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
               CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

int64_t tree_attn_workspace_bytes(int sms)
{
    const int64_t a = attn_rows_workspace_floats(sms), b = attn_tiles_workspace_floats(sms);
    return kUnitBytes + 4 * (a > b ? a : b);
}

cudaError_t launch_tree_attn(const AttnParams &p, int D, int kind, int sms, cudaStream_t s, bool pdl)
{
    // Rows that share a key/value head in the average request (of T / R tokens,
    // padding included): up to 32 are one unit of the streaming kernel; more go to
    // the 128-row tiles.  Measured, us, streaming kernel against tiles:
    //   heads of         32 on 8 of 128               64 on 8 of 64
    //   fp16, 1 request of 30001 places
    //     32 rows         36.6     39.2                25.0     26.6
    //     48 rows         43.4     43.0                31.5     27.9
    //   fp16, 16 requests of 4000
    //     32 rows         56.4     62.1                35.8     41.5
    //     48 rows         84.7     64.8                58.6     43.1
    //   8-bit, 1 request of 30001
    //     32 rows         35.9     40.0                25.6     34.0
    //     48 rows         51.0     41.6                36.9     34.6
    //   8-bit, 16 requests of 4000
    //     32 rows         57.2     86.1                41.1     62.0
    //     48 rows         97.7     88.3                70.3     63.4
    // The average says nothing of a batch that mixes single tokens and chunks of
    // prompts, and one kernel then takes both: 127 single tokens over 4096 places
    // and 512 tokens behind 8192, 559 us (8-bit 690) on the kernel chosen, 465 (829)
    // on the other, as two calls 316 + 79 (184 + 111); 63 and 1500 tokens 282 (493),
    // 581 (656), as two calls 165 + 85 (99 + 127).  A choice for each request would
    // have to be made on the device, where the lengths are; it is not built, and
    // include/qmv.h tells callers to make two calls.
    const int64_t rows = (p.T + p.R - 1) / p.R * p.group;
    if (rows <= 32) return launch_attn_rows(p, D, kind, rows, sms, s, pdl);
    return launch_attn_tiles(p, D, kind, sms, s, pdl);
}

}  // namespace qmv
