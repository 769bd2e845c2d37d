// tree_api.cu -- the C ABI of include/dspark_tree.h: argument checks, the
// handle's device memory, and the launches.
#include <cudaTypedefs.h>
#include <cuda_runtime.h>
#include <math.h>

#include <algorithm>
#include <new>

#include "../../include/dspark_tree.h"
#include "tree_common.cuh"

using namespace dspark::tree;

struct dspark_tree {
  int device = 0;
  int sm_count = 0;
  dspark_tree_config cfg{};
  int* status = nullptr;          // and after it a count a worker (AttendArgs::arrived)
  void* parts = nullptr;          // attend's workspace
  float* part_o = nullptr;
  float2* part_ml = nullptr;
  int4* part_of = nullptr;
  int part_rows = 0;
  uint32_t ready = 0;             // e2m1 kernels that have been launched (few4_launch)
  PFN_cuTensorMapEncodeTiled_v12000 encode = nullptr;
};

namespace {

int cuda_code(cudaError_t e) {
  if (e == cudaSuccess) return DSPARK_OK;
  return e == cudaErrorMemoryAllocation ? DSPARK_ENOMEM : DSPARK_ECUDA;
}

size_t status_bytes(const dspark_tree* h) { return (1 + kFew4Workers * h->sm_count) * sizeof(int); }

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

bool stride_ok(int64_t s, int es) { return s >= 0 && s <= ((int64_t)1 << 40) && s * es % 16 == 0; }

// Zeroes device memory before it returns, on a stream of its own: a memset alone is
// not waited for by the host, and kernels on streams of all kinds come after it.
cudaError_t clear(void* p, size_t bytes) {
  cudaStream_t s = nullptr;
  cudaError_t e = cudaStreamCreateWithFlags(&s, cudaStreamNonBlocking);
  if (e != cudaSuccess) return e;
  e = cudaMemsetAsync(p, 0, bytes, s);
  if (e == cudaSuccess) e = cudaStreamSynchronize(s);
  const cudaError_t d = cudaStreamDestroy(s);
  return e != cudaSuccess ? e : d;
}

// The handle's device is current while a call runs; the caller's is afterwards.
class OnDevice {
 public:
  explicit OnDevice(const dspark_tree* h) {
    int now = 0;
    if (cudaGetDevice(&now) != cudaSuccess) return;
    ok_ = now == h->device || cudaSetDevice(h->device) == cudaSuccess;
    if (ok_ && now != h->device) before_ = now;
  }
  ~OnDevice() {
    if (before_ >= 0) cudaSetDevice(before_);
  }
  OnDevice(const OnDevice&) = delete;
  OnDevice& operator=(const OnDevice&) = delete;
  int code() const { return ok_ ? DSPARK_OK : DSPARK_ECUDA; }

 private:
  bool ok_ = false;
  int before_ = -1;
};

int make_cache(const dspark_tree* h, const dspark_tree_cache* c, CacheView* out) {
  if (!c || !c->k || !c->v) return DSPARK_EINVAL;
  const bool e2m1 = c->type == DSPARK_TYPE_E2M1, scaled = e2m1 || c->type == DSPARK_TYPE_E4M3;
  if (c->type != h->cfg.type && !scaled) return DSPARK_EINVAL;
  const int es = scaled ? 1 : 2;
  if (scaled && (!c->k_scale || !c->v_scale || h->cfg.head_dim % (e2m1 ? 32 : 16)))
    return DSPARK_EINVAL;
  // bytes that a row's scales are read by at once: 8, 4 or 2
  const int64_t together = e2m1 ? h->cfg.head_dim / 16 & -(h->cfg.head_dim / 16) : 1;
  if (c->n_pages < 1 || c->n_pages >= ((int64_t)1 << 31) || c->page_size < 1) return DSPARK_EINVAL;
  if (!aligned16(c->k) || !aligned16(c->v)) return DSPARK_EINVAL;
  for (int v = 0; v < 2; ++v) {
    const int64_t* st = v ? c->v_stride : c->k_stride;
    const int64_t* ss = v ? c->v_scale_stride : c->k_scale_stride;
    for (int i = 0; i < 3; ++i) {
      if (!stride_ok(st[i], es)) return DSPARK_EINVAL;
      if (scaled && (ss[i] < 0 || ss[i] > ((int64_t)1 << 40) || ss[i] % together))
        return DSPARK_EINVAL;
      // pages and slots lie within 2 GB strides (see Rows); heads may be further apart
      if (i < 2 && (st[i] * es >= ((int64_t)1 << 31) || (scaled && ss[i] >= ((int64_t)1 << 31))))
        return DSPARK_EINVAL;
    }
    if (scaled && reinterpret_cast<uintptr_t>(v ? c->v_scale : c->k_scale) % together)
      return DSPARK_EINVAL;
    out->x[v] = {static_cast<uint8_t*>(v ? c->v : c->k), st[2] * es, (uint32_t)(st[0] * es),
                 (uint32_t)(st[1] * es)};
    out->scale[v] = {nullptr, 0, 0, 0};
    if (scaled)
      out->scale[v] = {v ? c->v_scale : c->k_scale, ss[2], (uint32_t)ss[0], (uint32_t)ss[1]};
  }
  out->n_pages = c->n_pages;
  out->page = FastDiv::of(c->page_size);
  return DSPARK_OK;
}

Held held_as(const dspark_tree_cache* c) {
  return c->type == DSPARK_TYPE_E4M3 ? kE4M3 : c->type == DSPARK_TYPE_E2M1 ? kE2M1 : k16;
}

// Tiled-copy maps of a 16-bit cache whose pages cut a 128-key tile into one or
// two boxes.  With 64-slot pages, by maps / by 16-byte copies: 17 nodes over 131,000
// tokens 102 / 138 us, 64 requests of 64 nodes 402 / 479 us.  With 16-slot pages a
// tile would be 32 boxes of 2 KB, which took 6,000 cycles, twice the copies' time:
// those, and strides that a map does not take, have none.
void make_maps(const dspark_tree* h, const dspark_tree_cache* c, const CacheView& v, TileMaps* m) {
  m->rows = 0;
  const int page = c->page_size;
  if (held_as(c) != k16 || !h->encode) return;
  if (page % 128 != 0 && page != 64) return;
  const cuuint64_t dims[4] = {(cuuint64_t)h->cfg.head_dim, (cuuint64_t)page,
                              (cuuint64_t)h->cfg.kv_heads, (cuuint64_t)c->n_pages};
  const cuuint32_t box[4] = {64, (cuuint32_t)(page < 128 ? page : 128), 1, 1};
  const cuuint32_t one[4] = {1, 1, 1, 1};
  const CUtensorMapDataType type = c->type == DSPARK_TYPE_F16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16
                                                               : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
  for (int i = 0; i < 2; ++i) {
    const Rows& r = v.x[i];
    const cuuint64_t strides[3] = {r.slot, (cuuint64_t)r.head, r.page};
    for (int d = 0; d < 3; ++d)
      if (strides[d] == 0 || strides[d] >= ((cuuint64_t)1 << 40)) return;
    if (h->encode(i ? &m->v : &m->k, type, 4, r.p, dims, strides, box, one,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                  CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
      return;
  }
  m->rows = (int)box[1];
}

int make_batch(const dspark_tree_batch* b, int page_size, bool rows, BatchView* out) {
  if (!b || b->B < 0 || (rows && b->N < 0)) return DSPARK_EINVAL;
  if (b->B == 0 || (rows && b->N == 0)) {
    out->B = 0;
    return DSPARK_OK;
  }
  if (!b->pages || !b->start || (rows && !b->first)) return DSPARK_EINVAL;
  if (b->max_pages < 1 || b->pages_stride < 0) return DSPARK_EINVAL;
  const int64_t max_pos = (int64_t)b->max_pages * page_size;
  if (max_pos >= ((int64_t)1 << 31)) return DSPARK_EINVAL;
  out->pages = b->pages;
  out->start = b->start;
  out->first = b->first;
  out->pages_stride = b->pages_stride;
  // a tile of keys past the last position still has a 32-bit place
  out->max_pos = max_pos < DSPARK_TREE_MAX_LENGTH ? max_pos : DSPARK_TREE_MAX_LENGTH;
  out->B = b->B;
  out->N = rows ? b->N : 0;
  return DSPARK_OK;
}

int make_rotation(const dspark_tree* h, const dspark_tree_rotation* r, int N, RotateArgs* a) {
  if (!r || N < 0) return DSPARK_EINVAL;
  const int D = h->cfg.head_dim, R = r->rotary_dim;
  if (D % 16 || R < 0 || R > D || R % 16 || (R > 0 && !r->turns)) return DSPARK_EINVAL;
  if (!isfinite(r->eps) || r->eps < 0.f || !aligned16(r->q_norm) || !aligned16(r->k_norm))
    return DSPARK_EINVAL;
  a->turns = r->turns;
  a->q_norm = r->q_norm;
  a->k_norm = r->k_norm;
  a->eps = r->eps;
  // fp32 loses squares below 2^-149: nothing beside a sum of 2^-80, or beside an eps of 2^-60
  a->least = r->eps < 0x1p-60f ? 0x1p-80f : 0.f;
  a->inv_dim = 1.f / (float)D;
  a->pairs = r->interleaved != 0;
  a->N = N;
  a->Hq = h->cfg.q_heads;
  a->Hkv = h->cfg.kv_heads;
  a->D = D;
  a->R = R;
  a->status = h->status;
  return DSPARK_OK;
}

bool source(RotateArgs* a, int i, const void* x, const int64_t* stride) {
  if (!x || !stride || !aligned16(x) || !stride_ok(stride[0], 2) || !stride_ok(stride[1], 2)) return false;
  a->src[i] = static_cast<const uint8_t*>(x);
  a->src_row[i] = stride[0] * 2;
  a->src_head[i] = stride[1] * 2;
  return true;
}

}  // namespace

extern "C" {

int dspark_tree_create(const dspark_tree_config* cfg, dspark_tree_t* out) {
  if (out) *out = nullptr;
  if (!cfg || !out) return DSPARK_EINVAL;
  if (cfg->kv_heads < 1 || cfg->q_heads < cfg->kv_heads || cfg->q_heads % cfg->kv_heads ||
      cfg->q_heads > 65535)
    return DSPARK_EINVAL;
  if (cfg->head_dim < 8 || cfg->head_dim % 8 || cfg->head_dim > DSPARK_TREE_MAX_HEAD_DIM)
    return DSPARK_EINVAL;
  if (cfg->type != DSPARK_TYPE_BF16 && cfg->type != DSPARK_TYPE_F16) return DSPARK_EINVAL;
  if (cfg->max_requests < 1 || cfg->max_requests > DSPARK_TREE_MAX_REQUESTS ||
      cfg->max_nodes < 1 || cfg->max_nodes > DSPARK_TREE_MAX_NODES)
    return DSPARK_EINVAL;
  int dev = 0, major = 0, minor = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return cuda_code(e);
  if (major != 10 || minor != 3) return DSPARK_EUNSUPPORTED;
  dspark_tree* h = new (std::nothrow) dspark_tree();
  if (!h) return DSPARK_ENOMEM;
  h->device = dev;
  h->sm_count = sms;
  h->cfg = *cfg;
  // two parts a worker: the item it finishes for an earlier one, and the one it
  // leaves to a later; as much as any of the kernels needs
  const int G = cfg->q_heads / cfg->kv_heads;
  const int64_t rows = (int64_t)cfg->max_nodes * G;
  h->part_rows = rows >= kGroupRows ? kGroupRows : (int)((rows + 31) / 32 * 32);
  const size_t n_parts = (size_t)2 * sms;
  size_t n_rows = n_parts * h->part_rows;
  if (cfg->head_dim % 32 == 0) n_rows = std::max(n_rows, (size_t)kFew4PartRows * sms);   // e2m1 may come
  const size_t o_bytes = n_rows * padded_dim(cfg->head_dim) * sizeof(float);
  const size_t ml_bytes = n_rows * sizeof(float2);
  e = cudaMalloc(&h->parts, o_bytes + ml_bytes + n_parts * sizeof(int4));
  if (e == cudaSuccess) {
    uint8_t* p = static_cast<uint8_t*>(h->parts);
    h->part_o = reinterpret_cast<float*>(p);
    h->part_ml = reinterpret_cast<float2*>(p + o_bytes);
    h->part_of = reinterpret_cast<int4*>(p + o_bytes + ml_bytes);
    e = cudaMalloc(&h->status, status_bytes(h));
  }
  if (e == cudaSuccess) e = clear(h->status, status_bytes(h));
  if (e == cudaSuccess) {
    void* fn = nullptr;
    cudaDriverEntryPointQueryResult found = cudaDriverEntryPointSymbolNotFound;
    e = cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault,
                                         &found);
    if (e == cudaSuccess && found == cudaDriverEntryPointSuccess)
      h->encode = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(fn);
  }
  if (e == cudaSuccess) e = attend_setup(cfg->type == DSPARK_TYPE_F16, cfg->head_dim);
  if (e == cudaSuccess) e = few_setup(cfg->type == DSPARK_TYPE_F16, cfg->head_dim);
  if (e != cudaSuccess) {
    dspark_tree_destroy(h);
    return cuda_code(e);
  }
  *out = h;
  return DSPARK_OK;
}

int dspark_tree_write(dspark_tree_t h, const dspark_tree_cache* cache,
                      const dspark_tree_batch* batch, const void* k, const int64_t* k_stride,
                      const void* v, const int64_t* v_stride, void* stream) {
  if (!h) return DSPARK_EINVAL;
  RowsArgs a{};
  const OnDevice on(h);
  int rc = on.code();
  if (rc == DSPARK_OK) rc = make_cache(h, cache, &a.c);
  if (rc == DSPARK_OK) rc = make_batch(batch, cache->page_size, true, &a.b);
  if (rc != DSPARK_OK) return rc;
  if (a.b.B == 0) return DSPARK_OK;
  if (!k || !v || !k_stride || !v_stride || !aligned16(k) || !aligned16(v)) return DSPARK_EINVAL;
  for (int i = 0; i < 2; ++i)
    if (!stride_ok(k_stride[i], 2) || !stride_ok(v_stride[i], 2)) return DSPARK_EINVAL;
  for (int i = 0; i < 2; ++i) {
    a.src[i] = static_cast<const uint8_t*>(i ? v : k);
    a.src_row[i] = (i ? v_stride : k_stride)[0] * 2;
    a.src_head[i] = (i ? v_stride : k_stride)[1] * 2;
  }
  a.Hkv = h->cfg.kv_heads;
  a.kv2 = FastDiv::of(2 * a.Hkv);
  a.D = h->cfg.head_dim;
  a.status = h->status;
  return cuda_code(write_launch(a, h->cfg.type == DSPARK_TYPE_F16, held_as(cache), h->sm_count,
                                static_cast<cudaStream_t>(stream)));
}

int dspark_tree_read(dspark_tree_t h, const dspark_tree_cache* cache,
                     const dspark_tree_batch* batch, void* out_k, void* out_v, void* stream) {
  if (!h) return DSPARK_EINVAL;
  RowsArgs a{};
  const OnDevice on(h);
  int rc = on.code();
  if (rc == DSPARK_OK) rc = make_cache(h, cache, &a.c);
  if (rc == DSPARK_OK) rc = make_batch(batch, cache->page_size, true, &a.b);
  if (rc != DSPARK_OK) return rc;
  if (a.b.B == 0) return DSPARK_OK;
  if (!out_k || !out_v || !aligned16(out_k) || !aligned16(out_v)) return DSPARK_EINVAL;
  a.out[0] = static_cast<uint16_t*>(out_k);
  a.out[1] = static_cast<uint16_t*>(out_v);
  a.Hkv = h->cfg.kv_heads;
  a.kv2 = FastDiv::of(2 * a.Hkv);
  a.D = h->cfg.head_dim;
  a.status = h->status;
  return cuda_code(read_launch(a, h->cfg.type == DSPARK_TYPE_F16, held_as(cache), h->sm_count,
                               static_cast<cudaStream_t>(stream)));
}

int dspark_tree_keep(dspark_tree_t h, const dspark_tree_cache* cache,
                     const dspark_tree_batch* batch, const int32_t* path, int64_t path_stride,
                     int max_path, const int32_t* count, void* stream) {
  if (!h) return DSPARK_EINVAL;
  KeepArgs a{};
  const OnDevice on(h);
  int rc = on.code();
  if (rc == DSPARK_OK) rc = make_cache(h, cache, &a.c);
  if (rc == DSPARK_OK) rc = make_batch(batch, cache->page_size, false, &a.b);
  if (rc != DSPARK_OK) return rc;
  if (max_path < 0 || max_path > DSPARK_TREE_MAX_NODES) return DSPARK_EINVAL;
  if (a.b.B == 0 || max_path == 0) return DSPARK_OK;
  if (!path || !count || path_stride < 0) return DSPARK_EINVAL;
  a.path = path;
  a.count = count;
  a.path_stride = path_stride;
  a.max_path = max_path;
  a.Hkv = h->cfg.kv_heads;
  const Held held = held_as(cache);
  a.scale_bytes = held == kE4M3 ? 1 : held == kE2M1 ? h->cfg.head_dim / 16 : 0;
  a.row_bytes = held == kE2M1 ? h->cfg.head_dim / 2 : h->cfg.head_dim * (held == kE4M3 ? 1 : 2);
  a.status = h->status;
  return cuda_code(keep_launch(a, static_cast<cudaStream_t>(stream)));
}

int dspark_tree_attend(dspark_tree_t h, const dspark_tree_cache* cache,
                       const dspark_tree_batch* batch, const void* q, const int64_t* q_stride,
                       const uint32_t* mask, int64_t mask_stride, int mask_words, float scale,
                       float softcap, void* out, float* lse, void* stream) {
  if (!h) return DSPARK_EINVAL;
  AttendArgs a{};
  const OnDevice on(h);
  int rc = on.code();
  if (rc == DSPARK_OK) rc = make_cache(h, cache, &a.c);
  if (rc == DSPARK_OK) rc = make_batch(batch, cache->page_size, true, &a.b);
  if (rc != DSPARK_OK) return rc;
  if (!isfinite(scale) || !isfinite(softcap) || softcap < 0.f) return DSPARK_EINVAL;
  if (a.b.B > h->cfg.max_requests) return DSPARK_EINVAL;
  if (mask && (mask_words < 1 || mask_stride < 0)) return DSPARK_EINVAL;
  if (a.b.B == 0) return DSPARK_OK;
  if (!q || !q_stride || !out || !aligned16(q) || !aligned16(out)) return DSPARK_EINVAL;
  if (!stride_ok(q_stride[0], 2) || !stride_ok(q_stride[1], 2)) return DSPARK_EINVAL;
  a.q = static_cast<const uint8_t*>(q);
  a.q_row = q_stride[0] * 2;
  a.q_head = q_stride[1] * 2;
  a.mask = mask;
  a.mask_stride = mask_stride;
  // no more than nodes need, so that the bits of a row are a small number
  constexpr int kWords = (DSPARK_TREE_MAX_NODES + 31) / 32;
  a.mask_words = !mask ? 0 : mask_words < kWords ? mask_words : kWords;
  a.scale = scale;
  a.softcap = softcap;
  a.out = static_cast<uint16_t*>(out);
  a.lse = lse;
  a.Hq = h->cfg.q_heads;
  a.Hkv = h->cfg.kv_heads;
  a.G = a.Hq / a.Hkv;
  a.D = h->cfg.head_dim;
  a.max_nodes = h->cfg.max_nodes;
  a.group = FastDiv::of(a.G);
  a.n_cta = h->sm_count;
  a.part_o = h->part_o;
  a.part_ml = h->part_ml;
  a.part_of = h->part_of;
  a.part_rows = h->part_rows;
  a.arrived = h->status + 1;
  a.status = h->status;
  // Few rows a cached head on average: the kernels that have tiles of 16 of them (any
  // number of rows is right in either).  16 requests of 300 to 6,000 tokens, 8 heads,
  // us here / there.  16-slot pages, 16-bit: 4 rows 56 / 67, 16 rows 57 / 67, 20 rows
  // 96 / 67 (K and V read twice); e4m3, which the other kernel has to convert through
  // shared memory: 4 rows 42 / 65, 16 rows 44 / 66, 20 rows 70 / 66.  64-slot pages,
  // which the other kernel takes by tiled copies, 16-bit: 16 rows 56 / 55, 20 rows
  // 95 / 56; e4m3: 16 rows 43 / 66.
  const bool few = (int64_t)a.b.N * a.G <= (int64_t)16 * a.b.B;
  if (held_as(cache) == kE2M1) {
    a.f16 = h->cfg.type == DSPARK_TYPE_F16;
    // Items of 32 rows where the others have 16.  8 heads of 128, 300 to 6,000 tokens, bf16, keys
    // alike, here / there: 16 requests (56,874 keys) over 16-slot pages 17 rows 59 / 66 us, 24 rows
    // 59 / 66, 32 rows 62 / 66, over 64-slot ones 58 / 66, 58 / 66, 61 / 66; 128 requests 359 / 390,
    // 365 / 390, 378 / 391 and 347, 349, 365.  With one key in 50 eight times the others, which moves
    // maxima here, 24 rows 63 / 66 and 384 / 390, 32 rows 66 / 66 and 397 / 391 (32 requests 124 /
    // 119), in f16 66 / 71 and 398 / 415.  Weights are f16 here, eight times as fine as bf16 there.
    const bool few4 = (int64_t)a.b.N * a.G <= (int64_t)32 * a.b.B;
    return cuda_code(few4 ? few4_launch(a, &h->ready, static_cast<cudaStream_t>(stream))
                         : attend4_launch(a, a.f16, &h->ready, static_cast<cudaStream_t>(stream)));
  }
  if (few)
    return cuda_code(few_launch(a, h->cfg.type == DSPARK_TYPE_F16,
                                cache->type == DSPARK_TYPE_E4M3,
                                static_cast<cudaStream_t>(stream)));
  TileMaps maps;
  make_maps(h, cache, a.c, &maps);
  return cuda_code(attend_launch(a, maps, h->cfg.type == DSPARK_TYPE_F16,
                                 cache->type == DSPARK_TYPE_E4M3,
                                 static_cast<cudaStream_t>(stream)));
}

int dspark_tree_rotate(dspark_tree_t h, const dspark_tree_rotation* rotation, const int32_t* position,
                       int N, const void* q, const int64_t* q_stride, const void* k,
                       const int64_t* k_stride, void* out_q, void* out_k, void* stream) {
  if (!h) return DSPARK_EINVAL;
  RotateArgs a{};
  const OnDevice on(h);
  int rc = on.code();
  if (rc == DSPARK_OK) rc = make_rotation(h, rotation, N, &a);
  if (rc != DSPARK_OK) return rc;
  if (N == 0) return DSPARK_OK;
  if (!position || !out_q || !out_k || !aligned16(out_q) || !aligned16(out_k)) return DSPARK_EINVAL;
  if (!source(&a, 0, q, q_stride) || !source(&a, 1, k, k_stride)) return DSPARK_EINVAL;
  a.position = position;
  a.out_q = static_cast<uint16_t*>(out_q);
  a.out_k = static_cast<uint16_t*>(out_k);
  return cuda_code(rotate_launch(a, false, h->cfg.type == DSPARK_TYPE_F16, k16, h->sm_count,
                                 static_cast<cudaStream_t>(stream)));
}

int dspark_tree_place(dspark_tree_t h, const dspark_tree_cache* cache, const int32_t* slot,
                      const dspark_tree_rotation* rotation, const int32_t* position, int N,
                      const void* q, const int64_t* q_stride, const void* k, const int64_t* k_stride,
                      const void* v, const int64_t* v_stride, void* out_q, void* stream) {
  if (!h) return DSPARK_EINVAL;
  RotateArgs a{};
  const OnDevice on(h);
  int rc = on.code();
  if (rc == DSPARK_OK) rc = make_cache(h, cache, &a.c);
  if (rc == DSPARK_OK) rc = make_rotation(h, rotation, N, &a);
  if (rc != DSPARK_OK) return rc;
  a.slots = cache->n_pages * cache->page_size;
  if (a.slots >= ((int64_t)1 << 31)) return DSPARK_EINVAL;
  if (N == 0) return DSPARK_OK;
  if (!position || !slot || !out_q || !aligned16(out_q)) return DSPARK_EINVAL;
  if (!source(&a, 0, q, q_stride) || !source(&a, 1, k, k_stride) || !source(&a, 2, v, v_stride))
    return DSPARK_EINVAL;
  a.position = position;
  a.slot = slot;
  a.out_q = static_cast<uint16_t*>(out_q);
  return cuda_code(rotate_launch(a, true, h->cfg.type == DSPARK_TYPE_F16, held_as(cache),
                                 h->sm_count, static_cast<cudaStream_t>(stream)));
}

int dspark_tree_status(dspark_tree_t h, void* stream) {
  if (!h) return DSPARK_EINVAL;
  const OnDevice on(h);
  if (on.code() != DSPARK_OK) return on.code();
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  int st = 0;
  cudaError_t e = cudaMemcpyAsync(&st, h->status, sizeof(int), cudaMemcpyDeviceToHost, s);
  if (e == cudaSuccess) e = cudaMemsetAsync(h->status, 0, status_bytes(h), s);
  if (e == cudaSuccess) e = cudaStreamSynchronize(s);
  return e == cudaSuccess ? st : cuda_code(e);
}

int dspark_tree_destroy(dspark_tree_t h) {
  if (!h) return DSPARK_EINVAL;
  const OnDevice on(h);
  const int rc = on.code() != DSPARK_OK ? on.code() : cuda_code(cudaDeviceSynchronize());
  if (h->status) cudaFree(h->status);
  if (h->parts) cudaFree(h->parts);
  delete h;
  return rc;
}

}  // extern "C"
