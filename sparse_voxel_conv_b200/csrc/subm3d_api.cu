// C ABI of the submanifold 3x3x3 sparse convolution (include/subm3d.h):
// argument checks, workspace sizing, the map handle, and kernel dispatch.
// No device memory is allocated here; every buffer belongs to the caller.
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdlib>
#include <cstring>
#include <memory>
#include <mutex>
#include <new>

#include "internal.h"
#include "subm3d.h"

// The library's device error word: set to 1 by a forward kernel whose bounded
// wait ran out; read and cleared by subm3d_device_status().
static __device__ int32_t g_subm3d_error_word;

struct subm3d_map {
  const int32_t* nbr;
  const uint32_t* tile_mask;
  const uint32_t* status_word;
  const int32_t* pos;     // x-run position table
  const int32_t* et;      // E index table
  const int32_t* hdr;     // [runs, position tiles, positions, 0]
  int64_t ptile_max;      // position tiles reserved in the workspace
  const void* workspace;  // the build's workspace, laid out as `layout`
  subm3d::MapLayout layout;
  int64_t n;
  int32_t grid_dim;
  int32_t batch;
  cudaStream_t stream;
};

namespace {

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

// Testing knobs read from the environment at every call:
//   SUBM3D_TABLE_CAPACITY=<slots>  caps the hash table (and selects it), so that
//                                  a full table can be exercised;
//   SUBM3D_MAP_KIND=hash           uses the hash table even where the direct
//                                  or brick table would fit;
//   SUBM3D_MAP_KIND=brick|direct   uses that table wherever it fits (within
//                                  the direct table's size budget).
subm3d::MapOptions options_from_env() {
  subm3d::MapOptions o;
  const char* cap = std::getenv("SUBM3D_TABLE_CAPACITY");
  if (cap && *cap) o.forced_capacity = std::strtoull(cap, nullptr, 10);
  const char* kind = std::getenv("SUBM3D_MAP_KIND");
  if (kind && std::strcmp(kind, "hash") == 0) o.force_hash = true;
  if (kind && std::strcmp(kind, "brick") == 0) o.force_brick = true;
  if (kind && std::strcmp(kind, "direct") == 0) o.force_direct = true;
  return o;
}

// 1 when the current device is sm_100 (B200 class), 0 when it is not, -1 on error.
int device_is_sm100(int* device_out) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return -1;
  static std::mutex mu;
  static signed char cache[64];
  static bool init = false;
  std::lock_guard<std::mutex> lock(mu);
  if (!init) {
    std::memset(cache, -1, sizeof(cache));
    init = true;
  }
  if (device_out) *device_out = dev;
  if (dev >= 0 && dev < 64 && cache[dev] >= 0) return cache[dev];
  int major = 0, minor = 0;
  if (cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev) != cudaSuccess)
    return -1;
  const int ok = (major == 10 && minor == 0) ? 1 : 0;
  if (dev >= 0 && dev < 64) cache[dev] = static_cast<signed char>(ok);
  return ok;
}

// Limit of each pipeline wait inside the tensor-core kernels: 2 s, or the
// testing knob SUBM3D_WAIT_LIMIT_NS=<ns> (read at every call), with which a
// test makes the waits run out and checks the timeout path.
uint64_t wait_limit_from_env() {
  const char* v = std::getenv("SUBM3D_WAIT_LIMIT_NS");
  if (v && *v) {
    const unsigned long long ns = std::strtoull(v, nullptr, 10);
    if (ns > 0) return ns;
  }
  return 2000000000ull;
}

int32_t* device_error_word() {
  static std::mutex mu;
  static int32_t* addr[64] = {};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return nullptr;
  std::lock_guard<std::mutex> lock(mu);
  if (!addr[dev]) {
    void* p = nullptr;
    if (cudaGetSymbolAddress(&p, g_subm3d_error_word) != cudaSuccess) return nullptr;
    addr[dev] = static_cast<int32_t*>(p);
  }
  return addr[dev];
}

}  // namespace

extern "C" {

int32_t subm3d_abi_version(void) { return SUBM3D_ABI_VERSION; }

const char* subm3d_status_string(int32_t status) {
  switch (status) {
    case SUBM3D_OK: return "ok";
    case SUBM3D_E_INVALID: return "invalid argument";
    case SUBM3D_E_RANGE: return "coordinate out of range";
    case SUBM3D_E_DUPLICATE: return "duplicate coordinate";
    case SUBM3D_E_TABLE_FULL: return "hash table full";
    case SUBM3D_E_UNSUPPORTED: return "unsupported shape, alignment or device";
    case SUBM3D_E_CUDA: return "CUDA runtime error";
    case SUBM3D_E_TIMEOUT: return "device-side wait timed out";
    default: return "unknown status";
  }
}

size_t subm3d_map_workspace_bytes(int64_t n, int32_t grid_dim, int32_t batch) {
  subm3d::MapLayout lay;
  if (!subm3d::map_layout(n, grid_dim, batch, options_from_env(), &lay)) return 0;
  return lay.total;
}

subm3d_status subm3d_build_map(const int32_t* coords, int64_t n, int32_t grid_dim,
                               int32_t batch, int32_t* nbr, void* workspace,
                               size_t workspace_bytes, void* stream, subm3d_map** out_map) {
  if (!out_map) return SUBM3D_E_INVALID;
  *out_map = nullptr;
  if (n < 0 || !workspace) return SUBM3D_E_INVALID;
  if (n > 0 && (!coords || !nbr)) return SUBM3D_E_INVALID;
  subm3d::MapLayout lay;
  if (!subm3d::map_layout(n, grid_dim, batch, options_from_env(), &lay))
    return (grid_dim < 1 || batch < 1) ? SUBM3D_E_INVALID : SUBM3D_E_UNSUPPORTED;
  if (workspace_bytes < lay.total) return SUBM3D_E_INVALID;
  if (!aligned(coords, 16) || !aligned(nbr, 16) || !aligned(workspace, 256))
    return SUBM3D_E_INVALID;
  auto* h = new (std::nothrow) subm3d_map;
  if (!h) return SUBM3D_E_INVALID;
  auto* ws = static_cast<uint8_t*>(workspace);
  h->nbr = nbr;
  h->tile_mask = reinterpret_cast<const uint32_t*>(ws + lay.mask_off);
  h->status_word = reinterpret_cast<const uint32_t*>(ws + lay.status_off);
  const bool runs = lay.ptile_max > 0;
  h->pos = runs ? reinterpret_cast<const int32_t*>(ws + lay.pos_off) : nullptr;
  h->et = runs ? reinterpret_cast<const int32_t*>(ws + lay.et_off) : nullptr;
  h->hdr = runs ? reinterpret_cast<const int32_t*>(ws + lay.hdr_off) : nullptr;
  h->ptile_max = lay.ptile_max;
  h->workspace = workspace;
  h->layout = lay;
  h->n = n;
  h->grid_dim = grid_dim;
  h->batch = batch;
  h->stream = static_cast<cudaStream_t>(stream);
  if (subm3d::launch_map_build(coords, n, grid_dim, batch, nbr, workspace, lay,
                               h->stream) != cudaSuccess) {
    delete h;
    return SUBM3D_E_CUDA;
  }
  *out_map = h;
  return SUBM3D_OK;
}

subm3d_status subm3d_map_status(const subm3d_map* map) {
  if (!map) return SUBM3D_E_INVALID;
  uint32_t word = 0;
  if (cudaMemcpyAsync(&word, map->status_word, sizeof(word), cudaMemcpyDeviceToHost,
                      map->stream) != cudaSuccess ||
      cudaStreamSynchronize(map->stream) != cudaSuccess)
    return SUBM3D_E_CUDA;
  if (word & subm3d::kErrRange) return SUBM3D_E_RANGE;
  if (word & subm3d::kErrDuplicate) return SUBM3D_E_DUPLICATE;
  if (word & subm3d::kErrTableFull) return SUBM3D_E_TABLE_FULL;
  return SUBM3D_OK;
}

const int32_t* subm3d_map_nbr(const subm3d_map* map) { return map ? map->nbr : nullptr; }
const uint32_t* subm3d_map_tile_mask(const subm3d_map* map) {
  return map ? map->tile_mask : nullptr;
}
int64_t subm3d_map_size(const subm3d_map* map) { return map ? map->n : -1; }
int32_t subm3d_map_table(const subm3d_map* map) {
  if (!map) return -1;
  switch (map->layout.kind) {
    case subm3d::MapKind::kDirect: return SUBM3D_TABLE_DIRECT;
    case subm3d::MapKind::kBrick: return SUBM3D_TABLE_BRICK;
    default: return SUBM3D_TABLE_HASH;
  }
}
void subm3d_map_destroy(subm3d_map* map) { delete map; }

namespace {

bool overlaps(const void* p, size_t p_bytes, const void* q, size_t q_bytes) {
  const auto* a = static_cast<const uint8_t*>(p);
  const auto* b = static_cast<const uint8_t*>(q);
  return a < b + q_bytes && b < a + p_bytes;
}

// Kernel choice for a map with an x-run layout: the x-run kernel when Cin >= 48.
// It does tensor work on every position (voxels and pads) for all 27 offsets,
// the per-offset kernel on every voxel for the offsets present in its 256-row
// tile but with ~3x the gathered bytes; timed with the GELU epilogue on three
// sets (x-runs of 9.3 and 4.0 voxels, 1.22 and 1.50 positions per voxel) at 64
// and 128 input and output channels, the x-run kernel was faster in every case,
// by 14% (4 x 256^3 shells, 64 -> 128) to 2.1x; with a partial last chunk it is
// 2.0-2.3x faster at 48 and 80 input channels on the headline set and 1.4x at
// 96 -> 64 on the decoder-stack set, but at 32 channels (half of its only
// chunk zeros) it is no faster than the per-offset kernel, which keeps Cin < 48.
// Testing knob SUBM3D_FORWARD_KERNEL (read at every call): "gather" takes the
// per-offset kernel even where the x-run kernel applies.
bool prefer_gather() {
  const char* knob = std::getenv("SUBM3D_FORWARD_KERNEL");
  return knob && std::strcmp(knob, "gather") == 0;
}

// The forward of every entry point: map may be null (nbr-only callers), in
// which case the x-run kernel is not available.
subm3d_status forward_impl(const subm3d_map* map, const int32_t* nbr, const uint32_t* tile_mask,
                           int64_t n, const void* feats, const void* weight, const void* bias,
                           const void* residual, void* out, int32_t cin, int32_t cout,
                           subm3d_dtype dtype, int32_t flip, subm3d_act act, void* stream) {
  if (n < 0 || cin < 1 || cout < 1) return SUBM3D_E_INVALID;
  if (dtype != SUBM3D_F32 && dtype != SUBM3D_BF16) return SUBM3D_E_INVALID;
  if (act != SUBM3D_ACT_NONE && act != SUBM3D_ACT_GELU && act != SUBM3D_ACT_SILU)
    return SUBM3D_E_INVALID;
  if (n > 0 && (!nbr || !feats || !weight || !out)) return SUBM3D_E_INVALID;
  if (n >= 0x7FFFFFFFll) return SUBM3D_E_UNSUPPORTED;
  if (n == 0) return SUBM3D_OK;
  const size_t esz = dtype == SUBM3D_BF16 ? 2 : 4;
  const size_t out_bytes = static_cast<size_t>(n) * cout * esz;
  if (overlaps(feats, static_cast<size_t>(n) * cin * esz, out, out_bytes))
    return SUBM3D_E_INVALID;  // out overlaps feats
  if (residual && residual != out && overlaps(residual, out_bytes, out, out_bytes))
    return SUBM3D_E_INVALID;  // a residual partly overlapping out would race
  auto s = static_cast<cudaStream_t>(stream);
  const int flip01 = flip ? 1 : 0;
  subm3d::Epilogue epi;
  epi.bias = bias;
  epi.residual = residual;
  epi.act = act == SUBM3D_ACT_GELU ? subm3d::kActGelu
                                   : (act == SUBM3D_ACT_SILU ? subm3d::kActSilu : subm3d::kActNone);
  if (dtype == SUBM3D_F32) {
    if (!aligned(nbr, 4) || !aligned(feats, 4) || !aligned(weight, 4) || !aligned(out, 4) ||
        (tile_mask && !aligned(tile_mask, 4)) || !aligned(bias, 4) || !aligned(residual, 4))
      return SUBM3D_E_INVALID;
    return subm3d::launch_forward_f32(nbr, tile_mask, n, static_cast<const float*>(feats),
                                      static_cast<const float*>(weight), static_cast<float*>(out),
                                      cin, cout, flip01, epi, s) == cudaSuccess
               ? SUBM3D_OK
               : SUBM3D_E_CUDA;
  }
  if (cin % 16 != 0 || cout % 16 != 0) return SUBM3D_E_UNSUPPORTED;
  if (!aligned(nbr, 16) || !aligned(feats, 16) || !aligned(weight, 16) || !aligned(out, 16) ||
      (tile_mask && !aligned(tile_mask, 4)) || !aligned(bias, 2) || !aligned(residual, 16))
    return SUBM3D_E_UNSUPPORTED;
  const int sm100 = device_is_sm100(nullptr);
  if (sm100 < 0) return SUBM3D_E_CUDA;
  if (sm100 == 0) return SUBM3D_E_UNSUPPORTED;
  subm3d::DeviceCtl ctl;
  ctl.err_word = device_error_word();
  if (!ctl.err_word) return SUBM3D_E_CUDA;
  ctl.wait_limit_ns = wait_limit_from_env();
  cudaError_t e;
  if (map && map->pos && cin >= 48 && !prefer_gather())  // cin % 16 == 0 (checked above)
    e = subm3d::launch_forward_bf16_runs(map->pos, map->et, map->layout.et_stride, map->hdr,
                                         map->ptile_max, feats,
                                         weight, out, cin, cout, flip01, epi, ctl, s);
  else
    e = subm3d::launch_forward_bf16(nbr, tile_mask, n, feats, weight, out, cin, cout, flip01, epi,
                                    ctl, s);
  if (e == cudaErrorNotSupported) return SUBM3D_E_UNSUPPORTED;
  return e == cudaSuccess ? SUBM3D_OK : SUBM3D_E_CUDA;
}

}  // namespace

subm3d_status subm3d_forward(const int32_t* nbr, const uint32_t* tile_mask, int64_t n,
                             const void* feats, const void* weight, void* out, int32_t cin,
                             int32_t cout, subm3d_dtype dtype, int32_t flip, subm3d_act act,
                             void* stream) {
  return forward_impl(nullptr, nbr, tile_mask, n, feats, weight, nullptr, nullptr, out, cin, cout,
                      dtype, flip, act, stream);
}

subm3d_status subm3d_map_run_layout(const subm3d_map* map, const int32_t** pos,
                                    const int32_t** etable, const int32_t** header) {
  if (!map || !pos || !etable || !header) return SUBM3D_E_INVALID;
  if (!map->pos) return SUBM3D_E_UNSUPPORTED;
  *pos = map->pos;
  *etable = map->et;
  *header = map->hdr;
  return SUBM3D_OK;
}

subm3d_status subm3d_forward_map(const subm3d_map* map, const void* feats, const void* weight,
                                 void* out, int32_t cin, int32_t cout, subm3d_dtype dtype,
                                 int32_t flip, subm3d_act act, void* stream) {
  if (!map) return SUBM3D_E_INVALID;
  return forward_impl(map, map->nbr, map->tile_mask, map->n, feats, weight, nullptr, nullptr, out,
                      cin, cout, dtype, flip, act, stream);
}

subm3d_status subm3d_forward_fused(const subm3d_map* map, const void* feats, const void* weight,
                                   const void* bias, const void* residual, void* out, int32_t cin,
                                   int32_t cout, subm3d_dtype dtype, int32_t flip, subm3d_act act,
                                   void* stream) {
  if (!map) return SUBM3D_E_INVALID;
  return forward_impl(map, map->nbr, map->tile_mask, map->n, feats, weight, bias, residual, out,
                      cin, cout, dtype, flip, act, stream);
}

subm3d_status subm3d_backward_data(const subm3d_map* map, const void* dy, const void* weight,
                                   void* weight_t, void* dx, int32_t cin, int32_t cout,
                                   subm3d_dtype dtype, int32_t flip, void* stream) {
  if (!map || cin < 1 || cout < 1) return SUBM3D_E_INVALID;
  if (dtype != SUBM3D_F32 && dtype != SUBM3D_BF16) return SUBM3D_E_INVALID;
  if (map->n == 0) return SUBM3D_OK;
  if (!dy || !weight || !weight_t || !dx) return SUBM3D_E_INVALID;
  const size_t esz = dtype == SUBM3D_BF16 ? 2 : 4;
  const size_t w_bytes = static_cast<size_t>(cout) * 27 * cin * esz;
  if (overlaps(weight, w_bytes, weight_t, w_bytes)) return SUBM3D_E_INVALID;
  if (!aligned(weight, esz) || !aligned(weight_t, 16)) return SUBM3D_E_INVALID;
  auto s = static_cast<cudaStream_t>(stream);
  if (subm3d::launch_transpose_weight(weight, weight_t, cout, cin, dtype == SUBM3D_BF16, s) !=
      cudaSuccess)
    return SUBM3D_E_CUDA;
  // dx = forward of dy with W^T (Cout -> Cin) and the opposite orientation
  return forward_impl(map, map->nbr, map->tile_mask, map->n, dy, weight_t, nullptr, nullptr, dx,
                      cout, cin, dtype, flip ? 0 : 1, SUBM3D_ACT_NONE, stream);
}

subm3d_status subm3d_backward_weight(const subm3d_map* map, const void* feats, const void* dy,
                                     float* dweight, int32_t cin, int32_t cout,
                                     subm3d_dtype dtype, int32_t flip, void* stream) {
  if (!map || cin < 1 || cout < 1 || !dweight) return SUBM3D_E_INVALID;
  if (dtype != SUBM3D_F32 && dtype != SUBM3D_BF16) return SUBM3D_E_INVALID;
  const int64_t n = map->n;
  if (n > 0 && (!feats || !dy)) return SUBM3D_E_INVALID;
  const size_t esz = dtype == SUBM3D_BF16 ? 2 : 4;
  if (!aligned(feats, esz) || !aligned(dy, esz) || !aligned(dweight, 4)) return SUBM3D_E_INVALID;
  const size_t dw_bytes = static_cast<size_t>(cout) * 27 * cin * 4;
  if (n > 0 && (overlaps(dweight, dw_bytes, feats, static_cast<size_t>(n) * cin * esz) ||
                overlaps(dweight, dw_bytes, dy, static_cast<size_t>(n) * cout * esz)))
    return SUBM3D_E_INVALID;
  auto s = static_cast<cudaStream_t>(stream);
  if (n > 0 && dtype == SUBM3D_BF16 && map->pos && cin % 16 == 0 && cout % 16 == 0 &&
      aligned(feats, 16) && aligned(dy, 16) && aligned(dweight, 16) && device_is_sm100(nullptr) == 1) {
    subm3d::DeviceCtl ctl;
    ctl.err_word = device_error_word();
    if (!ctl.err_word) return SUBM3D_E_CUDA;
    ctl.wait_limit_ns = wait_limit_from_env();
    return subm3d::launch_wgrad_bf16_runs(map->pos, map->et, map->layout.et_stride, map->hdr,
                                          feats, dy, dweight, cin,
                                          cout, flip ? 1 : 0, ctl, s) == cudaSuccess
               ? SUBM3D_OK
               : SUBM3D_E_CUDA;
  }
  int device = 0, sms = 0;
  if (cudaGetDevice(&device) != cudaSuccess ||
      cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, device) != cudaSuccess)
    return SUBM3D_E_CUDA;
  return subm3d::launch_wgrad(map->nbr, n, feats, dy, dweight, cin, cout, flip ? 1 : 0,
                              dtype == SUBM3D_BF16, sms, s) ==
                 cudaSuccess
             ? SUBM3D_OK
             : SUBM3D_E_CUDA;
}

size_t subm3d_expand_workspace_bytes(int64_t n) {
  if (n < 0 || n >= (int64_t(1) << 28)) return 0;
  return subm3d::expand_layout(n).bytes;
}

subm3d_status subm3d_expand(const int32_t* coords, const void* feats, const uint8_t* mask,
                            int64_t n, int32_t channels_out, subm3d_dtype dtype,
                            subm3d_expand_mode mode, int32_t* out_coords, void* out_feats,
                            void* workspace, size_t workspace_bytes, int64_t* out_count,
                            void* stream) {
  if (!out_count || n < 0 || channels_out < 1) return SUBM3D_E_INVALID;
  *out_count = 0;
  if (dtype != SUBM3D_F32 && dtype != SUBM3D_BF16) return SUBM3D_E_INVALID;
  if (mode != SUBM3D_EXPAND_SUBDIVIDE && mode != SUBM3D_EXPAND_UPSAMPLE &&
      mode != SUBM3D_EXPAND_CHANNEL2SPATIAL)
    return SUBM3D_E_INVALID;
  if ((mode == SUBM3D_EXPAND_SUBDIVIDE && mask) || (mode == SUBM3D_EXPAND_UPSAMPLE && !mask))
    return SUBM3D_E_INVALID;
  if (n >= (int64_t(1) << 28)) return SUBM3D_E_UNSUPPORTED;
  if (n == 0) return SUBM3D_OK;
  if (!coords || !feats || !out_coords || !out_feats || !workspace) return SUBM3D_E_INVALID;
  if (workspace_bytes < subm3d::expand_layout(n).bytes) return SUBM3D_E_INVALID;
  const size_t esz = dtype == SUBM3D_BF16 ? 2 : 4;
  if (!aligned(coords, 16) || !aligned(out_coords, 16) || !aligned(workspace, 256) ||
      !aligned(feats, esz) || !aligned(out_feats, esz))
    return SUBM3D_E_INVALID;
  const bool slice = mode == SUBM3D_EXPAND_CHANNEL2SPATIAL;
  const int64_t out_row = static_cast<int64_t>(channels_out) * esz;
  const int64_t in_row = slice ? 8 * out_row : out_row;
  const cudaError_t e = subm3d::launch_expand(
      coords, feats, mask, n, in_row, out_row, slice, mode == SUBM3D_EXPAND_SUBDIVIDE, out_coords,
      out_feats, workspace, out_count, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? SUBM3D_OK : SUBM3D_E_CUDA;
}

size_t subm3d_pool_workspace_bytes(int64_t n, int32_t grid_dim, int32_t batch) {
  if (n < 0 || grid_dim < 1 || grid_dim > 65535 || batch < 1 || batch > 65535) return 0;
  const subm3d::PoolLayout l = subm3d::pool_layout(n, grid_dim, batch);
  if (l.cells > (int64_t(1) << 30)) return 0;
  return l.bytes;
}

subm3d_status subm3d_pool(const subm3d_map* fine, const int32_t* coords, const void* feats,
                          int32_t channels, subm3d_dtype dtype, subm3d_pool_mode mode,
                          int32_t* out_coords, void* out_feats, void* workspace,
                          size_t workspace_bytes, int64_t* out_count, void* stream) {
  if (!fine || !out_count || channels < 1) return SUBM3D_E_INVALID;
  *out_count = 0;
  if (dtype != SUBM3D_F32 && dtype != SUBM3D_BF16) return SUBM3D_E_INVALID;
  if (mode != SUBM3D_POOL_MAX && mode != SUBM3D_POOL_MEAN && mode != SUBM3D_POOL_SPATIAL2CHANNEL)
    return SUBM3D_E_INVALID;
  const int64_t n = fine->n;
  const size_t need = subm3d_pool_workspace_bytes(n, fine->grid_dim, fine->batch);
  if (need == 0) return SUBM3D_E_UNSUPPORTED;
  if (!workspace || workspace_bytes < need || !aligned(workspace, 256)) return SUBM3D_E_INVALID;
  if (n > 0 && (!coords || !feats || !out_coords || !out_feats)) return SUBM3D_E_INVALID;
  const size_t esz = dtype == SUBM3D_BF16 ? 2 : 4;
  if (!aligned(coords, 16) || !aligned(out_coords, 16) || !aligned(feats, esz) ||
      !aligned(out_feats, esz))
    return SUBM3D_E_INVALID;
  const cudaError_t e = subm3d::launch_pool(
      fine->layout, fine->workspace, fine->grid_dim, fine->batch, coords, n, feats, channels,
      dtype == SUBM3D_BF16, static_cast<int>(mode), out_coords, out_feats, workspace, out_count,
      static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? SUBM3D_OK : SUBM3D_E_CUDA;
}

namespace {

bool valid_dtype(int d) { return d == SUBM3D_F32 || d == SUBM3D_BF16; }
bool valid_act(int a) {
  return a == SUBM3D_ACT_NONE || a == SUBM3D_ACT_GELU || a == SUBM3D_ACT_SILU;
}
size_t dtype_bytes(int d) { return d == SUBM3D_BF16 ? 2 : 4; }

constexpr int32_t kMaxNormChannels = 1 << 24;
constexpr int64_t kMaxElements = int64_t(1) << 46;  // keeps every byte count inside 64 bits

// The SM count of the current device, 0 on error.
int sm_count() {
  static std::mutex mu;
  static int cache[64] = {};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return 0;
  std::lock_guard<std::mutex> lock(mu);
  if (dev >= 0 && dev < 64 && cache[dev] > 0) return cache[dev];
  int sms = 0;
  if (cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return 0;
  if (dev >= 0 && dev < 64) cache[dev] = sms;
  return sms;
}

// A buffer of a call: its bytes and whether the call writes it.
struct Span {
  uintptr_t begin, end;
  bool written;
};

// Whether a written buffer shares a byte with any other one.
bool clash(Span* spans, size_t count) {
  std::sort(spans, spans + count,
            [](const Span& a, const Span& b) { return a.begin < b.begin; });
  uintptr_t any_end = 0, written_end = 0;
  for (size_t i = 0; i < count; ++i) {
    if (spans[i].begin == spans[i].end) continue;
    if (spans[i].begin < written_end || (spans[i].written && spans[i].begin < any_end))
      return true;
    any_end = std::max(any_end, spans[i].end);
    if (spans[i].written) written_end = std::max(written_end, spans[i].end);
  }
  return false;
}
Span span(const void* p, int64_t bytes, bool written) {
  const auto b = reinterpret_cast<uintptr_t>(p);
  return p ? Span{b, b + static_cast<uintptr_t>(bytes), written} : Span{0, 0, false};
}

// Bytes from the first element of n rows, `stride` elements apart, to the last.
int64_t rows_bytes(int64_t n, int64_t stride, int64_t width, size_t esz) {
  return n > 0 ? ((n - 1) * stride + width) * static_cast<int64_t>(esz) : 0;
}

// Turns per unit of position of each pair.  The thread's last table is kept, told by the
// numbers that it was made from: its exponentials are a microsecond of a short call.
struct RotaryTable {
  double theta = 0.0;
  int32_t axis_pairs[subm3d::kRotaryMaxAxes] = {};
  double turns[subm3d::kRotaryMaxPairs];
};
const RotaryTable& rotary_table(double theta, const int32_t (&axis_pairs)[subm3d::kRotaryMaxAxes]) {
  static thread_local RotaryTable t;
  if (t.theta == theta && std::equal(axis_pairs, axis_pairs + subm3d::kRotaryMaxAxes, t.axis_pairs))
    return t;
  const double log_theta = std::log(theta);
  int used = 0;
  for (int32_t pairs : axis_pairs)
    for (int32_t j = 0; j < pairs; ++j)
      t.turns[used++] = std::exp(-log_theta * j / pairs) / 6.283185307179586476925;
  t.theta = theta;
  std::copy(axis_pairs, axis_pairs + subm3d::kRotaryMaxAxes, t.axis_pairs);
  return t;
}

subm3d_status of(cudaError_t e) { return e == cudaSuccess ? SUBM3D_OK : SUBM3D_E_CUDA; }

}  // namespace

subm3d_status subm3d_layer_norm(const void* x, int64_t n, int32_t channels, int64_t x_stride,
                                subm3d_dtype dtype, const void* weight, const void* bias,
                                subm3d_dtype affine_dtype, float eps, subm3d_act act, void* y,
                                float* mean, float* rstd, void* stream) {
  if (n < 0 || channels < 1 || x_stride < channels || !valid_dtype(dtype) || !valid_act(act) ||
      !valid_dtype(affine_dtype) || (affine_dtype == SUBM3D_BF16 && dtype != SUBM3D_BF16) ||
      !(eps >= 0.0f) || std::isinf(eps) || !mean != !rstd)
    return SUBM3D_E_INVALID;
  if (channels > kMaxNormChannels || (n > 0 && x_stride > kMaxElements / n))
    return SUBM3D_E_UNSUPPORTED;
  if (n == 0) return SUBM3D_OK;
  if (!x || !y) return SUBM3D_E_INVALID;
  const size_t esz = dtype_bytes(dtype), asz = dtype_bytes(affine_dtype);
  if (!aligned(x, esz) || !aligned(y, esz) || !aligned(weight, asz) || !aligned(bias, asz) ||
      !aligned(mean, 4) || !aligned(rstd, 4))
    return SUBM3D_E_INVALID;
  const bool in_place = y == x && (n == 1 || x_stride == channels);
  Span spans[] = {span(in_place ? nullptr : x, rows_bytes(n, x_stride, channels, esz), false),
                  span(weight, channels * static_cast<int64_t>(asz), false),
                  span(bias, channels * static_cast<int64_t>(asz), false),
                  span(y, rows_bytes(n, channels, channels, esz), true),
                  span(mean, 4 * n, true),
                  span(rstd, 4 * n, true)};
  if (clash(spans, 6)) return SUBM3D_E_INVALID;
  subm3d::LayerNormArgs a;
  a.x = x;
  a.weight = weight;
  a.bias = bias;
  a.y = y;
  a.mean = mean;
  a.rstd = rstd;
  a.n = n;
  a.x_stride = x_stride;
  a.c = channels;
  a.act = act;
  a.eps = eps;
  a.bf16 = dtype == SUBM3D_BF16;
  a.affine_bf16 = affine_dtype == SUBM3D_BF16;
  const int sms = sm_count();
  if (sms == 0) return SUBM3D_E_CUDA;
  return of(subm3d::launch_layer_norm(a, sms, static_cast<cudaStream_t>(stream)));
}

size_t subm3d_layer_norm_workspace_bytes(int64_t n, int32_t channels) {
  if (n < 0 || channels < 1 || channels > kMaxNormChannels) return 0;
  const int64_t chunks = subm3d::layer_norm_chunks(n, channels);
  return chunks > 1 ? static_cast<size_t>(chunks) * 2 * channels * 4 : 0;
}

subm3d_status subm3d_layer_norm_backward(
    const void* dy, int64_t dy_stride, const void* x, int64_t x_stride, int64_t n,
    int32_t channels, subm3d_dtype dtype, const float* mean, const float* rstd,
    const void* weight, const void* bias, subm3d_dtype affine_dtype, subm3d_act act, void* dx,
    float* dweight, float* dbias, void* workspace, size_t workspace_bytes, void* stream) {
  if (n < 0 || channels < 1 || x_stride < channels || dy_stride < channels ||
      !valid_dtype(dtype) || !valid_act(act) || !valid_dtype(affine_dtype) ||
      (affine_dtype == SUBM3D_BF16 && dtype != SUBM3D_BF16))
    return SUBM3D_E_INVALID;
  if (channels > kMaxNormChannels ||
      (n > 0 && (x_stride > kMaxElements / n || dy_stride > kMaxElements / n)))
    return SUBM3D_E_UNSUPPORTED;
  if (!aligned(dweight, 4) || !aligned(dbias, 4)) return SUBM3D_E_INVALID;
  auto s = static_cast<cudaStream_t>(stream);
  const int64_t c4 = static_cast<int64_t>(channels) * 4;
  if (n == 0) {
    if (dweight && cudaMemsetAsync(dweight, 0, c4, s) != cudaSuccess) return SUBM3D_E_CUDA;
    if (dbias && cudaMemsetAsync(dbias, 0, c4, s) != cudaSuccess) return SUBM3D_E_CUDA;
    return SUBM3D_OK;
  }
  if (!dx && !dweight && !dbias) return SUBM3D_OK;
  const bool sums = dweight || dbias;
  const size_t need = sums ? subm3d_layer_norm_workspace_bytes(n, channels) : 0;
  if (!dy || !x || !mean || !rstd || (need && !workspace)) return SUBM3D_E_INVALID;
  const size_t esz = dtype_bytes(dtype), asz = dtype_bytes(affine_dtype);
  if (workspace_bytes < need || (need && !aligned(workspace, 16)) || !aligned(dy, esz) ||
      !aligned(x, esz) || !aligned(dx, esz) || !aligned(weight, asz) || !aligned(bias, asz) ||
      !aligned(mean, 4) || !aligned(rstd, 4))
    return SUBM3D_E_INVALID;
  Span spans[] = {span(dy, rows_bytes(n, dy_stride, channels, esz), false),
                  span(x, rows_bytes(n, x_stride, channels, esz), false),
                  span(mean, 4 * n, false),
                  span(rstd, 4 * n, false),
                  span(weight, channels * static_cast<int64_t>(asz), false),
                  span(bias, channels * static_cast<int64_t>(asz), false),
                  span(dx, rows_bytes(n, channels, channels, esz), true),
                  span(dweight, c4, true),
                  span(dbias, c4, true),
                  span(need ? workspace : nullptr, static_cast<int64_t>(need), true)};
  if (clash(spans, 10)) return SUBM3D_E_INVALID;
  subm3d::LayerNormGradArgs a;
  a.dy = dy;
  a.x = x;
  a.mean = mean;
  a.rstd = rstd;
  a.weight = weight;
  a.bias = bias;
  a.dx = dx;
  a.dweight = dweight;
  a.dbias = dbias;
  a.partial = need ? static_cast<float*>(workspace) : nullptr;
  a.n = n;
  a.x_stride = x_stride;
  a.dy_stride = dy_stride;
  a.c = channels;
  a.act = act;
  a.bf16 = dtype == SUBM3D_BF16;
  a.affine_bf16 = affine_dtype == SUBM3D_BF16;
  const int sms = sm_count();
  if (sms == 0) return SUBM3D_E_CUDA;
  return of(subm3d::launch_layer_norm_grad(a, sms, s));
}

subm3d_status subm3d_rotary(const void* x, int64_t x_row, int64_t x_head, int64_t n,
                            int32_t heads, int32_t head_dim, subm3d_dtype dtype,
                            const void* positions, int32_t positions_f32, int64_t pos_stride,
                            int32_t axes, const int32_t* axis_pairs, double theta, int32_t halves,
                            int32_t inverse, void* y, int64_t y_row, int64_t y_head,
                            void* stream) {
  if (n < 0 || heads < 0 || head_dim < 2 || !valid_dtype(dtype) || axes < 1 ||
      axes > subm3d::kRotaryMaxAxes || !axis_pairs || !(theta > 0.0) || std::isinf(theta) ||
      x_row < 0 || x_head < 0 || y_row < 0 || y_head < 0 || pos_stride < 0)
    return SUBM3D_E_INVALID;
  if (head_dim % 2 != 0 || head_dim / 2 > subm3d::kRotaryMaxPairs) return SUBM3D_E_UNSUPPORTED;
  int64_t used = 0;
  for (int i = 0; i < axes; ++i) {
    if (axis_pairs[i] < 0 || axis_pairs[i] > head_dim / 2 - used) return SUBM3D_E_INVALID;
    used += axis_pairs[i];
  }
  if (n == 0 || heads == 0) return SUBM3D_OK;
  // rows and heads of y apart from each other (a row may hold its heads, or a head its rows)
  if ((heads > 1 && y_head < head_dim) || (n > 1 && y_row < head_dim)) return SUBM3D_E_INVALID;
  if (n > 1 && heads > 1 &&
      !(y_row >= (heads - 1) * y_head + head_dim || y_head >= (n - 1) * y_row + head_dim))
    return SUBM3D_E_INVALID;
  const int64_t most = kMaxElements / n / heads;
  if (x_row > most || x_head > most || y_row > most || y_head > most || pos_stride > most)
    return SUBM3D_E_UNSUPPORTED;
  const size_t esz = dtype_bytes(dtype);
  if (!x || !y || !positions || !aligned(x, esz) || !aligned(y, esz) || !aligned(positions, 4))
    return SUBM3D_E_INVALID;
  const bool in_place = y == x && (n == 1 || y_row == x_row) && (heads == 1 || y_head == x_head);
  const auto reach = [&](int64_t row, int64_t head, int64_t width, size_t size) {
    return ((n - 1) * row + (heads - 1) * head + width) * static_cast<int64_t>(size);
  };
  Span spans[] = {span(in_place ? nullptr : x, reach(x_row, x_head, head_dim, esz), false),
                  span(positions, ((n - 1) * pos_stride + axes) * 4, false),
                  span(y, reach(y_row, y_head, head_dim, esz), true)};
  if (clash(spans, 3)) return SUBM3D_E_INVALID;
  subm3d::RotaryArgs a;
  std::copy(axis_pairs, axis_pairs + axes, a.axis_pairs);
  const RotaryTable& table = rotary_table(theta, a.axis_pairs);
  std::copy(table.turns, table.turns + used, a.turns);
  a.x = x;
  a.y = y;
  a.pos = positions;
  a.n = n;
  a.x_row = x_row;
  a.x_head = x_head;
  a.y_row = y_row;
  a.y_head = y_head;
  a.pos_stride = pos_stride;
  a.heads = heads;
  a.head_dim = head_dim;
  a.axes = axes;
  a.pairs = static_cast<int32_t>(used);
  a.bf16 = dtype == SUBM3D_BF16;
  a.pos_f32 = positions_f32 != 0;
  a.halves = halves != 0;
  a.inverse = inverse != 0;
  const int sms = sm_count();
  if (sms == 0) return SUBM3D_E_CUDA;
  return of(subm3d::launch_rotary(a, sms, static_cast<cudaStream_t>(stream)));
}

extern "C++" {
namespace {

// Launches over `tensors` in lists of up to CAP.
template <int CAP>
cudaError_t adamw_lists(const subm3d_adamw_tensor* tensors, int32_t count,
                        const subm3d::AdamWStep& a, bool bits8, cudaStream_t stream) {
  subm3d::AdamWList<CAP> l;
  l.count = 0;
  int64_t blocks = 0;
  const auto flush = [&]() -> cudaError_t {
    cudaError_t e = cudaSuccess;
    if (l.count > 0)
      e = subm3d::launch_adamw(a, l, static_cast<uint32_t>(blocks), bits8, stream);
    l.count = 0;
    blocks = 0;
    return e;
  };
  for (int32_t i = 0; i < count; ++i) {
    const subm3d_adamw_tensor& t = tensors[i];
    if (t.n == 0) continue;
    const int64_t need = (t.n + subm3d::adamw_chunk() - 1) / subm3d::adamw_chunk();
    // a list's tensors are consecutive ones: their numbers count from the first
    if (l.count > 0 && (l.count == CAP || blocks + need > 0x7FFFFFFFll ||
                        l.first_tensor + l.count != i)) {
      const cudaError_t e = flush();
      if (e != cudaSuccess) return e;
    }
    if (l.count == 0) l.first_tensor = i;
    l.first_block[l.count] = static_cast<uint32_t>(blocks);
    const size_t state = bits8 ? 8 : 16;
    const bool whole = aligned(t.param, 16) && aligned(t.grad, 16) && aligned(t.master, 16) &&
                       aligned(t.exp_avg, state) && aligned(t.exp_avg_sq, state);
    l.tensors[l.count] = {t.param,
                          t.grad,
                          t.exp_avg,
                          t.exp_avg_sq,
                          static_cast<uint8_t*>(t.exp_avg_scale),
                          static_cast<uint8_t*>(t.exp_avg_sq_scale),
                          static_cast<float*>(t.master),
                          t.n,
                          whole};
    ++l.count;
    blocks += need;
  }
  return flush();
}

}  // namespace
}  // extern "C++"

subm3d_status subm3d_adamw(const subm3d_adamw_tensor* tensors, int32_t count,
                           const subm3d_adamw_step* step, void* stream) {
  if (count < 0 || (count > 0 && !tensors) || !step) return SUBM3D_E_INVALID;
  const subm3d_adamw_step& c = *step;
  const auto finite_from_0 = [](double v) { return v >= 0.0 && !std::isinf(v); };
  if (!valid_dtype(c.param_dtype) || !valid_dtype(c.grad_dtype) ||
      (c.state_bits != 32 && c.state_bits != 8) || !(c.beta1 >= 0.0 && c.beta1 < 1.0) ||
      !(c.beta2 >= 0.0 && c.beta2 < 1.0) || !finite_from_0(c.eps) ||
      !finite_from_0(c.weight_decay) || (!c.lr_device && !finite_from_0(c.lr)) ||
      (!c.step_device && c.step < 1) || !aligned(c.step_device, 4) || !aligned(c.lr_device, 4))
    return SUBM3D_E_INVALID;
  if (count == 0) return SUBM3D_OK;
  const size_t psz = dtype_bytes(c.param_dtype), gsz = dtype_bytes(c.grad_dtype);
  const bool bits8 = c.state_bits == 8;
  const size_t ssz = bits8 ? 1 : 4;
  constexpr int kSpans = 7;
  std::unique_ptr<Span[]> spans(new (std::nothrow) Span[static_cast<size_t>(count) * kSpans + 2]);
  if (!spans) return SUBM3D_E_INVALID;
  size_t k = 0;
  spans[k++] = span(c.step_device, 4, false);
  spans[k++] = span(c.lr_device, 4, false);
  for (int32_t i = 0; i < count; ++i) {
    const subm3d_adamw_tensor& t = tensors[i];
    if (t.n < 0) return SUBM3D_E_INVALID;
    if (t.n > (int64_t(1) << 40)) return SUBM3D_E_UNSUPPORTED;
    if (t.n == 0) continue;
    if (!t.param || !t.grad || !t.exp_avg || !t.exp_avg_sq ||
        (bits8 && (!t.exp_avg_scale || !t.exp_avg_sq_scale)))
      return SUBM3D_E_INVALID;
    if (!aligned(t.param, psz) || !aligned(t.grad, gsz) || !aligned(t.exp_avg, ssz) ||
        !aligned(t.exp_avg_sq, ssz) || !aligned(t.master, 4))
      return SUBM3D_E_INVALID;
    const int64_t blocks32 = bits8 ? (t.n + 31) / 32 : 0;
    spans[k++] = span(t.param, t.n * static_cast<int64_t>(psz), true);
    spans[k++] = span(t.grad, t.n * static_cast<int64_t>(gsz), false);
    spans[k++] = span(t.exp_avg, t.n * static_cast<int64_t>(ssz), true);
    spans[k++] = span(t.exp_avg_sq, t.n * static_cast<int64_t>(ssz), true);
    spans[k++] = span(bits8 ? t.exp_avg_scale : nullptr, blocks32, true);
    spans[k++] = span(bits8 ? t.exp_avg_sq_scale : nullptr, blocks32, true);
    spans[k++] = span(t.master, t.n * 4, true);
  }
  if (clash(spans.get(), k)) return SUBM3D_E_INVALID;
  subm3d::AdamWStep a = {};
  a.beta1 = static_cast<float>(c.beta1);
  a.one_beta1 = static_cast<float>(1.0 - c.beta1);
  a.beta2 = static_cast<float>(c.beta2);
  a.one_beta2 = static_cast<float>(1.0 - c.beta2);
  a.eps = static_cast<float>(c.eps);
  a.minus_zero = -0.0f;
  a.lr = c.lr;
  a.weight_decay = c.weight_decay;
  a.log_beta1 = std::log(c.beta1);
  a.log_beta2 = std::log(c.beta2);
  a.step = c.step;
  a.step_device = c.step_device;
  a.lr_device = c.lr_device;
  a.seed = c.seed;
  a.param_bf16 = c.param_dtype == SUBM3D_BF16;
  a.grad_bf16 = c.grad_dtype == SUBM3D_BF16;
  const double t = static_cast<double>(c.step);
  a.step_size = static_cast<float>(c.lr / -std::expm1(t * a.log_beta1));
  a.inv_sqrt_bc2 = static_cast<float>(1.0 / std::sqrt(-std::expm1(t * a.log_beta2)));
  a.decay = static_cast<float>(1.0 - c.lr * c.weight_decay);
  auto s = static_cast<cudaStream_t>(stream);
  return of(count <= subm3d::kAdamWFew
                ? adamw_lists<subm3d::kAdamWFew>(tensors, count, a, bits8, s)
                : adamw_lists<subm3d::kAdamWMany>(tensors, count, a, bits8, s));
}

subm3d_status subm3d_device_status(void* stream) {
  int32_t* err = device_error_word();
  if (!err) return SUBM3D_E_CUDA;
  auto s = static_cast<cudaStream_t>(stream);
  int32_t word = 0;
  const int32_t zero = 0;
  if (cudaMemcpyAsync(&word, err, sizeof(word), cudaMemcpyDeviceToHost, s) != cudaSuccess ||
      cudaMemcpyAsync(err, &zero, sizeof(zero), cudaMemcpyHostToDevice, s) != cudaSuccess ||
      cudaStreamSynchronize(s) != cudaSuccess)
    return SUBM3D_E_CUDA;
  return word ? SUBM3D_E_TIMEOUT : SUBM3D_OK;
}

}  // extern "C"
