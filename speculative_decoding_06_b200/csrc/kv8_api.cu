// C entry points of the 8-bit paged K/V cache: argument checks (all before any
// work is queued) and the handle.
#include <cuda.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstdarg>
#include <cstdio>
#include <new>

#include "../../include/spec.h"
#include "kv8.h"

using namespace spec;

struct spec_kv8 {
  spec_kv8_config cfg{};
  uint8_t* codes = nullptr;
  uint8_t* exps = nullptr;
  int device = 0;
  int sm_count = 148;
  int clusters[kKv8TcMaxChunks + 1] = {};  // of the tree kernel: see kv8_tree_configure
  int page_log2 = 4;
  CUtensorMap map;  // the codes as rows of 128 bytes, boxes of 16 rows, 128-byte swizzle
  char err[256] = "";
};

namespace {

int fail(spec_kv8* h, int code, const char* fmt, ...) {
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(h->err, sizeof(h->err), fmt, ap);
  va_end(ap);
  return code;
}

bool config_ok(const spec_kv8_config* c) {
  return c && c->n_layers >= 1 && c->n_kv_heads >= 1 && c->n_kv_heads <= 65535 && c->head_dim == kKv8Hd &&
         (c->page == 16 || c->page == 32 || c->page == 64 || c->page == 128) && c->n_pages >= 1 &&
         (int64_t)c->n_pages * c->page < ((int64_t)1 << 31) &&
         // rows of 128 codes are numbered in 32 bits
         (double)c->n_layers * 2 * c->n_pages * c->n_kv_heads * c->page < 2147483648.0;
}

size_t exp_bytes_of(const spec_kv8_config& c) {
  return (size_t)c.n_layers * 2 * c.n_pages * c.n_kv_heads;
}

// the cache's GPU has to be the current one
int check_device(spec_kv8* h) {
  int dev = -1;
  const cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return fail(h, SPEC_ERR_CUDA, "cudaGetDevice failed: %s", cudaGetErrorName(e));
  if (dev != h->device) return fail(h, SPEC_ERR_ARG, "the cache is on device %d, the current device is %d", h->device, dev);
  return SPEC_OK;
}

int check_layer(spec_kv8* h, int layer) {
  if (layer < 0 || layer >= h->cfg.n_layers)
    return fail(h, SPEC_ERR_ARG, "layer %d outside [0, %d)", layer, h->cfg.n_layers);
  return SPEC_OK;
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// strides of rows of 128 values: whole 16-byte units, not negative
bool stride_ok(int64_t s, int elem) { return s >= 0 && (s * elem) % 16 == 0 && s < ((int64_t)1 << 40); }

Kv8View view_of(const spec_kv8* h, int layer) {
  const spec_kv8_config& c = h->cfg;
  Kv8View v;
  const size_t ep = (size_t)c.n_pages * c.n_kv_heads;
  const size_t cp = ep * c.page * kKv8Hd;
  for (int p = 0; p < 2; ++p) {
    v.codes[p] = h->codes + (2 * (size_t)layer + p) * cp;
    v.exps[p] = h->exps + (2 * (size_t)layer + p) * ep;
  }
  for (int p = 0; p < 2; ++p) v.row0[p] = (int)((2 * (size_t)layer + p) * ep * c.page);
  v.n_pages = c.n_pages;
  v.page = c.page;
  v.page_log2 = h->page_log2;
  v.hkv = c.n_kv_heads;
  return v;
}

bool encode_map(CUtensorMap* m, void* codes, uint64_t rows) {
  typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                    const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                    CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
  void* p = nullptr;
  cudaDriverEntryPointQueryResult q;
  if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) != cudaSuccess ||
      q != cudaDriverEntryPointSuccess)
    return false;
  const cuuint64_t dims[2] = {kKv8Hd, rows};
  const cuuint64_t strides[1] = {kKv8Hd};
  const cuuint32_t box[2] = {kKv8Hd, 16};
  const cuuint32_t estr[2] = {1, 1};
  return reinterpret_cast<EncodeTiledFn>(p)(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, codes, dims, strides, box, estr,
                                            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                                            CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
                                            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

int launched(spec_kv8* h, cudaError_t e, const char* what) {
  if (e == cudaSuccess) return SPEC_OK;
  return fail(h, SPEC_ERR_CUDA, "%s: %s (%s)", what, cudaGetErrorName(e), cudaGetErrorString(e));
}

}  // namespace

extern "C" {

size_t spec_kv8_code_bytes(const spec_kv8_config* cfg) {
  return config_ok(cfg) ? exp_bytes_of(*cfg) * cfg->page * kKv8Hd : 0;
}

size_t spec_kv8_exp_bytes(const spec_kv8_config* cfg) { return config_ok(cfg) ? exp_bytes_of(*cfg) : 0; }

int spec_kv8_open(const spec_kv8_config* cfg, void* codes, size_t code_bytes, void* exps, size_t exp_bytes,
                  spec_kv8** out) {
  if (!out) return SPEC_ERR_ARG;
  *out = nullptr;
  if (!config_ok(cfg) || !codes || !exps || (reinterpret_cast<uintptr_t>(codes) & 127u)) return SPEC_ERR_ARG;
  if (code_bytes < spec_kv8_code_bytes(cfg) || exp_bytes < spec_kv8_exp_bytes(cfg)) return SPEC_ERR_CAPACITY;
  // without a GPU the handle still checks its calls' arguments; they end in SPEC_ERR_CUDA
  int dev = -1, sms = 148, clusters[kKv8TcMaxChunks + 1] = {};
  if (cudaGetDevice(&dev) != cudaSuccess) {
    dev = -1;
    (void)cudaGetLastError();
  } else if (cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess ||
             kv8_plan_configure() != cudaSuccess || kv8_attention_configure(sms, clusters) != cudaSuccess) {
    return SPEC_ERR_CUDA;
  }
  spec_kv8* h = new (std::nothrow) spec_kv8;
  if (!h) return SPEC_ERR_CAPACITY;
  if (dev >= 0 && !encode_map(&h->map, codes, (uint64_t)spec_kv8_code_bytes(cfg) / kKv8Hd)) {
    delete h;
    return SPEC_ERR_CUDA;
  }
  h->cfg = *cfg;
  h->codes = static_cast<uint8_t*>(codes);
  h->exps = static_cast<uint8_t*>(exps);
  h->device = dev;
  h->sm_count = sms;
  for (int n = 0; n <= kKv8TcMaxChunks; ++n) h->clusters[n] = clusters[n];
  h->clusters[1] = sms;
  while ((1 << h->page_log2) < cfg->page) ++h->page_log2;
  *out = h;
  return SPEC_OK;
}

const char* spec_kv8_last_error(spec_kv8* h) { return h ? h->err : ""; }

void spec_kv8_close(spec_kv8* h) { delete h; }

int spec_kv8_plan(spec_kv8* h, const spec_kv8_plan_args* a, void* cuda_stream) {
  if (!h) return SPEC_ERR_ARG;
  if (!a || !a->lengths || !a->add || !a->tables || !a->ring || !a->state || !a->offsets || !a->lengths_out ||
      !a->state_out || !a->status || (!a->slots && a->max_rows > 0))
    return fail(h, SPEC_ERR_ARG, "null pointer");
  if (a->batch < 1 || a->n_seqs < 1 || a->max_blocks < 1 || a->max_rows < 0)
    return fail(h, SPEC_ERR_ARG, "batch, n_seqs and max_blocks must be positive, max_rows not negative");
  if (!a->seq_ids && a->batch > a->n_seqs)
    return fail(h, SPEC_ERR_ARG, "batch %d above n_seqs %d without seq_ids", a->batch, a->n_seqs);
  if (a->batch > kKv8MaxBatch || a->n_seqs > kKv8MaxSeqs)
    return fail(h, SPEC_ERR_CAPACITY, "batch above %d or n_seqs above %d", kKv8MaxBatch, kKv8MaxSeqs);
  if (a->max_rows > kKv8MaxRows) return fail(h, SPEC_ERR_CAPACITY, "max_rows above %d", kKv8MaxRows);
  if ((int64_t)a->max_blocks * h->cfg.page >= ((int64_t)1 << 31))
    return fail(h, SPEC_ERR_CAPACITY, "max_blocks * page has to be below 2^31");
  if (int rc = check_device(h)) return rc;
  return launched(h, launch_kv8_plan(*a, h->page_log2, h->cfg.n_pages, static_cast<cudaStream_t>(cuda_stream)),
                  "page plan");
}

int spec_kv8_append(spec_kv8* h, int layer, const spec_kv8_append_args* a, void* cuda_stream) {
  if (!h) return SPEC_ERR_ARG;
  if (int rc = check_layer(h, layer)) return rc;
  if (!a) return fail(h, SPEC_ERR_ARG, "null pointer");
  if (a->rows < 0 || a->n_src < 0) return fail(h, SPEC_ERR_ARG, "negative row count");
  if (!a->src_rows && a->n_src < a->rows)
    return fail(h, SPEC_ERR_ARG, "%d rows from %d source rows without src_rows", a->rows, a->n_src);
  if (a->dtype != SPEC_DTYPE_F32 && a->dtype != SPEC_DTYPE_BF16 && a->dtype != SPEC_DTYPE_F16)
    return fail(h, SPEC_ERR_ARG, "dtype must be SPEC_DTYPE_F32, SPEC_DTYPE_BF16 or SPEC_DTYPE_F16");
  if (a->rows > kKv8MaxRows) return fail(h, SPEC_ERR_CAPACITY, "more than %d rows", kKv8MaxRows);
  if (a->rows == 0) return SPEC_OK;
  if (!a->k || !a->v || !a->slots) return fail(h, SPEC_ERR_ARG, "null pointer");
  const int es = a->dtype == SPEC_DTYPE_F32 ? 4 : 2;
  if (!aligned16(a->k) || !aligned16(a->v) || !stride_ok(a->k_row_stride, es) || !stride_ok(a->k_head_stride, es) ||
      !stride_ok(a->v_row_stride, es) || !stride_ok(a->v_head_stride, es))
    return fail(h, SPEC_ERR_ARG, "k and v rows must be 16-byte aligned, with strides of whole 16-byte units");
  if (int rc = check_device(h)) return rc;
  return launched(h, launch_kv8_append(view_of(h, layer), *a, h->sm_count, static_cast<cudaStream_t>(cuda_stream)),
                  "append");
}

size_t spec_kv8_attention_workspace(spec_kv8* h, int batch, int n_q_heads, int max_nodes, int max_prefix) {
  if (!h || batch < 1 || n_q_heads < 1 || n_q_heads % h->cfg.n_kv_heads ||
      n_q_heads / h->cfg.n_kv_heads > kKv8MaxGroup || max_nodes < 1 || max_nodes > kKv8MaxNodes || max_prefix < 0 ||
      kv8_attention_need(view_of(h, 0), h->sm_count, batch, n_q_heads, max_nodes, max_prefix) == 0)
    return 0;
  return kv8_attention_workspace(view_of(h, 0), h->sm_count, batch, n_q_heads, max_nodes, max_prefix);
}

int spec_kv8_attention(spec_kv8* h, int layer, const spec_kv8_attention_args* a, void* cuda_stream) {
  if (!h) return SPEC_ERR_ARG;
  if (int rc = check_layer(h, layer)) return rc;
  if (!a) return fail(h, SPEC_ERR_ARG, "null pointer");
  if (a->batch < 1 || a->n_seqs < 1 || a->max_blocks < 1 || a->rows < 0 || a->n_q_heads < 1)
    return fail(h, SPEC_ERR_ARG, "batch, n_seqs, max_blocks and n_q_heads must be positive, rows not negative");
  if (!a->seq_ids && a->batch > a->n_seqs)
    return fail(h, SPEC_ERR_ARG, "batch %d above n_seqs %d without seq_ids", a->batch, a->n_seqs);
  if (a->n_q_heads % h->cfg.n_kv_heads) return fail(h, SPEC_ERR_ARG, "n_q_heads must be a multiple of n_kv_heads");
  if (a->n_q_heads / h->cfg.n_kv_heads > kKv8MaxGroup)
    return fail(h, SPEC_ERR_CAPACITY, "more than %d query heads per kv head", kKv8MaxGroup);
  if (a->dtype != SPEC_DTYPE_BF16 && a->dtype != SPEC_DTYPE_F16)
    return fail(h, SPEC_ERR_ARG, "dtype must be SPEC_DTYPE_BF16 or SPEC_DTYPE_F16");
  if (a->batch > 65535) return fail(h, SPEC_ERR_CAPACITY, "batch above 65535");
  if (a->max_nodes < 1 || a->max_nodes > kKv8MaxNodes)
    return fail(h, SPEC_ERR_CAPACITY, "max_nodes must be in [1, %d]", kKv8MaxNodes);
  if ((int64_t)a->max_blocks * h->cfg.page >= ((int64_t)1 << 31))
    return fail(h, SPEC_ERR_CAPACITY, "max_blocks * page has to be below 2^31");
  if (a->max_prefix < 0 || (int64_t)a->max_prefix > (int64_t)a->max_blocks * h->cfg.page)
    return fail(h, SPEC_ERR_CAPACITY, "max_prefix must be in [0, max_blocks * page]");
  if (!(a->scale >= 0.f) || !std::isfinite(a->scale)) return fail(h, SPEC_ERR_ARG, "scale must be finite and not negative");
  if ((a->k_new == nullptr) != (a->v_new == nullptr)) return fail(h, SPEC_ERR_ARG, "k_new and v_new go together");
  if (a->parents && !a->k_new) return fail(h, SPEC_ERR_ARG, "parents need k_new and v_new");
  if (a->fill & ~(SPEC_KV8_FILL_OUT | SPEC_KV8_FILL_LSE)) return fail(h, SPEC_ERR_ARG, "unknown bits in fill");
  if (!a->offsets || !a->tables || !a->lengths) return fail(h, SPEC_ERR_ARG, "null pointer");
  if (a->rows == 0) return SPEC_OK;
  if (!a->q || !a->out) return fail(h, SPEC_ERR_ARG, "null pointer");
  if (!aligned16(a->q) || !aligned16(a->out) || !aligned16(a->k_new) || !aligned16(a->v_new) ||
      !stride_ok(a->q_row_stride, 2) || !stride_ok(a->q_head_stride, 2) || !stride_ok(a->out_row_stride, 2) ||
      (a->k_new && (!stride_ok(a->k_row_stride, 2) || !stride_ok(a->k_head_stride, 2) ||
                    !stride_ok(a->v_row_stride, 2) || !stride_ok(a->v_head_stride, 2))))
    return fail(h, SPEC_ERR_ARG, "q, k_new, v_new and out rows must be 16-byte aligned, with strides of whole 16-byte units");
  if (a->out_row_stride < (int64_t)a->n_q_heads * kKv8Hd) return fail(h, SPEC_ERR_ARG, "out rows overlap");
  if (!a->workspace || !aligned16(a->workspace)) return fail(h, SPEC_ERR_ARG, "workspace is null or not 16-byte aligned");
  const size_t need = kv8_attention_need(view_of(h, 0), h->sm_count, a->batch, a->n_q_heads, a->max_nodes, a->max_prefix);
  if (need == 0) return fail(h, SPEC_ERR_CAPACITY, "more than %d row tiles (batch * n_kv_heads and more)", kKv8MaxGroups);
  if (a->workspace_bytes < need)
    return fail(h, SPEC_ERR_CAPACITY, "workspace too small");
  if (int rc = check_device(h)) return rc;
  spec_kv8_attention_args b = *a;
  if (b.scale == 0.f) b.scale = 0.08838834764831845f;  // 1 / sqrt(128)
  return launched(h, launch_kv8_attention(view_of(h, layer), h->map, b, h->clusters, static_cast<cudaStream_t>(cuda_stream)),
                  "attention");
}

}  // extern "C"
