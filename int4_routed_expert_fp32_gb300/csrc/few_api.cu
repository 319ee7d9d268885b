// Entry points of the routed experts of a few tokens: checks of arguments, the
// workspace, tensor maps (kernels in few.cu).
#include "few.cuh"

namespace moe {

namespace {

struct Few {
  FewArgs a;
  size_t bytes;
};

// Carves the workspace; with base == nullptr only the size is computed.
size_t carve(FewArgs* a, void* base) {
  size_t off = 0;
  auto take = [&](size_t bytes) -> void* {
    void* p = base && bytes ? static_cast<char*>(base) + off : nullptr;
    off += align_up(bytes, 256);
    return p;
  };
  const size_t T = a->T, P = T * a->k, D = a->D, H = a->H, L = a->L, S = a->S;
  const size_t tc = few_chunks(a->T, kFewRows / 2);
  a->n_counters = static_cast<int>(kFewFixed + P + D / 32 + (L ? H / 32 * tc : 0));
  a->counters = static_cast<int32_t*>(take(4 * static_cast<size_t>(a->n_counters)));
  a->scores = static_cast<float*>(take(a->router_w ? 4 * T * a->E : 0));
  a->keys = static_cast<uint32_t*>(take(a->router_w ? 4 * T * a->E : 0));
  a->x16 = static_cast<uint8_t*>(take(T * few_row_bytes(a->D)));
  a->x_unit = static_cast<float*>(take(4 * T));
  a->u_unit = static_cast<float*>(take(4 * T * (L / 16)));
  a->h16 = static_cast<uint8_t*>(take(P * few_row_bytes(a->I)));
  a->h_unit = static_cast<float*>(take(4 * P * (a->I / 16)));
  a->y = static_cast<float*>(take(4 * (P < kFewGroups ? P : kFewGroups) * T * D));
  a->hs = static_cast<uint16_t*>(take(4 * T * S));
  a->ys = static_cast<float*>(take(S ? 4 * T * H : 0));
  a->z = static_cast<uint16_t*>(take(4 * T * L));
  a->ssq = static_cast<float*>(take(4 * T * (L / 32)));
  a->yl = static_cast<float*>(take(L && S ? 4 * T * H : 0));
  return off;
}

bool sizes_ok(int T, int D, int E, int k, int I, int* rc) {
  *rc = MOE_ERR_INVALID;
  if (T < 0 || D <= 0 || E <= 0 || k <= 0 || I <= 0) return false;
  *rc = MOE_ERR_UNSUPPORTED;
  return T <= kFewTokens && D % 64 == 0 && I % 64 == 0 && D <= kFewWidth && I <= kFewWidth &&
         E <= kMaxExperts && k <= E && k <= kMaxTopK;
}

// Weights [n, rows, K] of 4 bits (words) or bf16 as [n, pieces, rows, 128 bytes]:
// 16 rows of a slot's pieces in one copy, of what is left over in the last slot of
// a row, and of the columns behind the last whole piece.
bool weight_maps(FewMaps* m, int which, const void* w, bool four, uint64_t K,
                 uint64_t rows, uint64_t n) {
  const uint64_t wide = four ? 256 : 64, row_bytes = four ? K / 2 : K * 2;
  const uint32_t unit = four ? 32 : 64, most = kFewColumns / 256;
  const uint64_t pieces = K / wide;
  const auto type = four ? CU_TENSOR_MAP_DATA_TYPE_INT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
  const uint64_t dims[4] = {unit, rows, pieces, n};
  const uint64_t strides[3] = {row_bytes, 128, row_bytes * rows};
  uint32_t box[4] = {unit, 16, most, 1};
  bool ok = true;
  if (pieces >= most)
    ok = encode_tensor_map(&m->full[which], type, 4, w, dims, strides, box,
                           CU_TENSOR_MAP_SWIZZLE_128B);
  box[2] = pieces % most;
  if (ok && box[2])
    ok = encode_tensor_map(&m->rest[which], type, 4, w, dims, strides, box,
                           CU_TENSOR_MAP_SWIZZLE_128B);
  if (ok && K % wide) {  // int4 only
    const uint64_t d3[3] = {K / 8, rows, n}, s3[2] = {row_bytes, row_bytes * rows};
    const uint32_t b3[3] = {unit, 16, 1};
    ok = encode_tensor_map(&m->tail[which], type, 3, w, d3, s3, b3, CU_TENSOR_MAP_SWIZZLE_128B);
  }
  return ok;
}

// bf16 rows of tokens [planes, T, K] as [planes, pieces, T, 128 bytes]: those of a pass
// over a slot of weights in one copy.
bool rows_map(CUtensorMap* m, const void* x, int T, int most, uint64_t K, uint64_t planes) {
  const uint64_t dims[4] = {64, static_cast<uint64_t>(T), K / 64, planes};
  const uint64_t strides[3] = {K * 2, 128, K * 2 * T};
  const uint32_t box[4] = {64, static_cast<uint32_t>(T < most ? T : most),
                           kFewColumns / 256, 1};
  return encode_tensor_map(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, x, dims, strides, box,
                           CU_TENSOR_MAP_SWIZZLE_128B);
}

// Their scales [n, rows, K / 32], 16 rows of what a slot needs.
bool scale_map(CUtensorMap* m, const void* s, uint64_t K, uint64_t rows, uint64_t n) {
  const uint64_t dims[3] = {K / kGroup, rows, n};
  const uint64_t strides[2] = {K / kGroup * 2, K / kGroup * 2 * rows};
  const uint32_t box[3] = {kFewColumns / kGroup, 16u, 1u};
  return encode_tensor_map(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, s, dims, strides, box,
                           CU_TENSOR_MAP_SWIZZLE_128B);
}

struct Experts {
  const int32_t* packed[3];  // gate, up, down
  const uint16_t* scale[3];
};

bool experts_ok(const Experts& w) {
  for (int i = 0; i < 3; ++i)
    if (!w.packed[i] || !w.scale[i] || !aligned(w.packed[i], 16) || !aligned(w.scale[i], 4))
      return false;
  return true;
}

struct Block {
  const void* p;
  size_t bytes;
};

// What the call reads of the experts.
void expert_blocks(const FewArgs& a, const Experts& w, Block* out) {
  const size_t n = static_cast<size_t>(a.E) * a.D * a.I;
  for (int i = 0; i < 3; ++i) {
    out[2 * i] = Block{w.packed[i], n / 2};
    out[2 * i + 1] = Block{w.scale[i], n / 16};
  }
}

int run(FewArgs a, const Experts& w, const moe_weights* layer, const Block* in, int n_in, void* ws,
        size_t ws_bytes, int stall_at, long long wait_ns, void* stream) {
  if (!aligned(ws, 256)) return MOE_ERR_INVALID;
  const size_t need = carve(&a, ws);
  if (ws_bytes < need) return MOE_ERR_WORKSPACE;
  const size_t out_bytes = static_cast<size_t>(a.T) * a.H * 2;
  for (int i = 0; i < n_in; ++i)
    if (overlap(in[i].p, in[i].bytes, a.out, out_bytes) || overlap(in[i].p, in[i].bytes, ws, need))
      return MOE_ERR_INVALID;
  if (overlap(a.out, out_bytes, ws, need)) return MOE_ERR_INVALID;
  a.stages = few_stages(a);
  if (a.stages < 2) return MOE_ERR_UNSUPPORTED;
  a.status = status_word();
  if (!a.status) return MOE_ERR_CUDA;
  a.wait_ns = wait_ns;
  a.stall_at = stall_at;
  for (int i = 0; i < 3; ++i) a.scale[i] = w.scale[i];
  // every expert's rows begin on 16 bytes where the first one's do: 16 rows of K / 16 bytes
  auto way = [](int K, bool on16) {
    return !on16 ? kScalesWords : K % 256 == 0 ? kScalesTma : K <= kFewColumns ? kScalesDense : kScalesWords;
  };
  a.tma_scale[0] = way(a.D, aligned(w.scale[0], 16) && aligned(w.scale[1], 16));
  a.tma_scale[1] = way(a.I, aligned(w.scale[2], 16));
  FewMaps m{};
  const uint64_t D = a.D, E = a.E, H = a.H, I = a.I, L = a.L, S = a.S;
  const struct {
    const void* w;
    const uint16_t* scale;
    uint64_t K, rows, n;
  } mats[kFewMatrices] = {{w.packed[0], a.tma_scale[0] == kScalesTma ? w.scale[0] : nullptr, D, I, E},
                          {w.packed[1], a.tma_scale[0] == kScalesTma ? w.scale[1] : nullptr, D, I, E},
                          {w.packed[2], a.tma_scale[1] == kScalesTma ? w.scale[2] : nullptr, I, D, E},
                          {L ? layer->lat_down : nullptr, nullptr, H, L, 1},
                          {L ? layer->lat_up : nullptr, nullptr, L, H, 1},
                          {S ? layer->shared_gate : nullptr, nullptr, H, S, 1},
                          {S ? layer->shared_up : nullptr, nullptr, H, S, 1},
                          {S ? layer->shared_down : nullptr, nullptr, S, H, 1}};
  for (int i = 0; i < kFewMatrices; ++i) {
    const auto& t = mats[i];
    if (t.w && !weight_maps(&m, i, t.w, i < 3, t.K, t.rows, t.n)) return MOE_ERR_CUDA;
    if (t.scale && !scale_map(&m.scale[i], t.scale, t.K, t.rows, t.n)) return MOE_ERR_CUDA;
  }
  if ((L || S) && !rows_map(&m.rows[0], a.x, a.T, kFewRows, H, 1)) return MOE_ERR_CUDA;
  if (S && !rows_map(&m.rows[1], a.hs, a.T, kFewRows / 2, S, 2)) return MOE_ERR_CUDA;
  if (L && !rows_map(&m.rows[2], a.z, a.T, kFewRows / 2, L, 2)) return MOE_ERR_CUDA;
  return launch_few(a, m, static_cast<cudaStream_t>(stream));
}

int experts_few(const uint16_t* x, const int32_t* topk_idx, const float* topk_w, int T, int D,
                int E, int k, int I, const Experts& w, uint16_t* out, void* ws, size_t ws_bytes,
                int stall_at, long long wait_ns, void* stream) {
  int rc;
  if (!sizes_ok(T, D, E, k, I, &rc)) return rc;
  if (T == 0) return MOE_OK;
  if (!x || !topk_idx || !topk_w || !out || !ws || !experts_ok(w)) return MOE_ERR_INVALID;
  if (!aligned(x, 16) || !aligned(out, 16) || !aligned(topk_idx, 4) || !aligned(topk_w, 4))
    return MOE_ERR_INVALID;
  FewArgs a{};
  a.x = x;
  a.topk_idx = topk_idx;
  a.topk_w = topk_w;
  a.out = out;
  a.T = T;
  a.H = a.D = D;
  a.E = E;
  a.k = k;
  a.I = I;
  Block in[9] = {{x, static_cast<size_t>(T) * D * 2},
                 {topk_idx, static_cast<size_t>(T) * k * 4},
                 {topk_w, static_cast<size_t>(T) * k * 4}};
  expert_blocks(a, w, in + 3);
  return run(a, w, nullptr, in, 9, ws, ws_bytes, stall_at, wait_ns, stream);
}

}  // namespace

}  // namespace moe

using namespace moe;

extern "C" size_t moe_experts_few_workspace_size(int T, int D, int E, int k, int I) {
  int rc;
  if (T <= 0 || !sizes_ok(T, D, E, k, I, &rc)) return 0;
  FewArgs a{};
  a.T = T;
  a.H = a.D = D;
  a.E = E;
  a.k = k;
  a.I = I;
  return carve(&a, nullptr);
}

extern "C" int moe_experts_few(const uint16_t* x, const int32_t* topk_idx, const float* topk_w,
                               int T, int D, int E, int k, int I, const int32_t* gate_packed,
                               const uint16_t* gate_scale, const int32_t* up_packed,
                               const uint16_t* up_scale, const int32_t* down_packed,
                               const uint16_t* down_scale, uint16_t* out, void* ws,
                               size_t ws_bytes, void* stream) {
  moe::Range range_("moe_experts_few");
  return experts_few(x, topk_idx, topk_w, T, D, E, k, I,
                     Experts{{gate_packed, up_packed, down_packed}, {gate_scale, up_scale, down_scale}},
                     out, ws, ws_bytes, -1, kDefaultWaitNs, stream);
}

extern "C" int moe_experts_few_stall_selftest(
    const uint16_t* x, const int32_t* topk_idx, const float* topk_w, int T, int D, int E, int k,
    int I, const int32_t* gate_packed, const uint16_t* gate_scale, const int32_t* up_packed,
    const uint16_t* up_scale, const int32_t* down_packed, const uint16_t* down_scale,
    int stall_stage, int64_t limit_ns, uint16_t* out, void* ws, size_t ws_bytes, void* stream) {
  moe::Range range_("moe_experts_few_stall_selftest");
  if (stall_stage < 0 || limit_ns < 1000 || limit_ns > 5000000000LL) return MOE_ERR_INVALID;
  return experts_few(x, topk_idx, topk_w, T, D, E, k, I,
                     Experts{{gate_packed, up_packed, down_packed}, {gate_scale, up_scale, down_scale}},
                     out, ws, ws_bytes, stall_stage, limit_ns, stream);
}

// The arguments of a layer call that need no pointers.
static bool layer_sizes(const moe_config* c, FewArgs* a, int* rc) {
  *rc = MOE_ERR_INVALID;
  if (!c || c->H <= 0 || c->L < 0 || c->I_shared < 0 || !(c->eps >= 0.f)) return false;
  if (!sizes_ok(c->T, c->L > 0 ? c->L : c->H, c->E, c->k, c->I, rc)) return false;
  *rc = MOE_ERR_UNSUPPORTED;
  if (c->H % 64 || c->I_shared % 64 || c->H > kFewWidth || c->I_shared > kFewWidth ||
      c->act_bits != 16)
    return false;
  a->T = c->T;
  a->H = c->H;
  a->E = c->E;
  a->k = c->k;
  a->I = c->I;
  a->L = c->L;
  a->D = c->L > 0 ? c->L : c->H;
  a->S = c->I_shared;
  a->renorm = c->renorm;
  a->eps = c->eps;
  return true;
}

extern "C" size_t moe_layer_few_workspace_size(const moe_config* cfg) {
  FewArgs a{};
  int rc;
  if (!layer_sizes(cfg, &a, &rc) || a.T == 0) return 0;
  static const float routed = 0.f;
  a.router_w = &routed;  // only whether there is one counts here
  return carve(&a, nullptr);
}

extern "C" int moe_layer_few(const moe_config* cfg, const moe_weights* w, const uint16_t* x,
                             uint16_t* out, void* ws, size_t ws_bytes, void* stream) {
  moe::Range range_("moe_layer_few");
  FewArgs a{};
  int rc;
  if (!layer_sizes(cfg, &a, &rc)) return rc;
  if (!w) return MOE_ERR_INVALID;
  if (a.T == 0) return MOE_OK;
  const Experts ex{{w->gate_packed, w->up_packed, w->down_packed},
                   {w->gate_scale, w->up_scale, w->down_scale}};
  if (!x || !out || !ws || !w->router_w || !w->router_bias || !experts_ok(ex))
    return MOE_ERR_INVALID;
  if (!aligned(x, 16) || !aligned(out, 16) || !aligned(w->router_w, 16) ||
      !aligned(w->router_bias, 4))
    return MOE_ERR_INVALID;
  if (a.L > 0 && (!w->lat_down || !w->lat_up || !aligned(w->lat_down, 16) ||
                  !aligned(w->lat_up, 16) || !aligned(w->lat_norm, 2)))
    return MOE_ERR_INVALID;
  if (a.S > 0 && (!w->shared_gate || !w->shared_up || !w->shared_down ||
                  !aligned(w->shared_gate, 16) || !aligned(w->shared_up, 16) ||
                  !aligned(w->shared_down, 16)))
    return MOE_ERR_INVALID;
  a.x = x;
  a.out = out;
  a.router_w = w->router_w;
  a.router_bias = w->router_bias;
  a.lat_norm = a.L > 0 ? w->lat_norm : nullptr;
  a.norm = a.lat_norm != nullptr;
  const size_t T = a.T, H = a.H, E = a.E, L = a.L, S = a.S;
  Block in[15] = {{x, T * H * 2},
                  {w->router_w, E * H * 4},
                  {w->router_bias, E * 4},
                  {w->lat_down, L * H * 2},
                  {w->lat_up, L * H * 2},
                  {a.lat_norm, a.norm ? L * 2 : 0},
                  {w->shared_gate, S * H * 2},
                  {w->shared_up, S * H * 2},
                  {w->shared_down, S * H * 2}};
  expert_blocks(a, ex, in + 9);
  return run(a, ex, w, in, 15, ws, ws_bytes, -1, kDefaultWaitNs, stream);
}
