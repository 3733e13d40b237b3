// fp8mm_loss.cu -- C entries of softmax cross entropy over an FP8 product and
// of its gradients.
#include "fp8mm_loss.cuh"
#include "fp8mm_rows_host.h"

#include <initializer_list>

namespace {

using namespace fp8mm_host;
using namespace fp8loss;

constexpr int64_t kPieceBytes = int64_t(1) << 30;   // of dz, and of the piece of B in fp16
constexpr int64_t kFewNorms = 8192;
constexpr int kLeastWidth = 128;                    // of a tile
constexpr int64_t kMostRows = INT32_MAX - 1024;     // of A and columns of B: tiles' coordinates are int

int64_t aligned(int64_t bytes) { return cdiv(bytes, 256) * 256; }

int check_problem(const void *A, const void *B, const float *sa, const float *sb, int scale_mode, int a_type, int b_type,
                  const void *bias, int bias_type, const int64_t *target, int64_t M, int64_t N, int64_t K)
{
    if ((scale_mode != FP8MM_SCALE_TENSOR && scale_mode != FP8MM_SCALE_ROWWISE) ||
        (a_type != FP8MM_TYPE_E4M3 && a_type != FP8MM_TYPE_E5M2) ||
        (b_type != FP8MM_TYPE_E4M3 && b_type != FP8MM_TYPE_E5M2) || !row_type_known(bias_type))
        return FP8MM_ERR_MODE;
    if (M < 0 || N < 1 || M > kMostRows || N > kMostRows || K < 16 || K % 16 != 0 || K > (int64_t(1) << 24))
        return FP8MM_ERR_SHAPE;
    // tiles of 256 x 256 and their K slices are counted in int
    if (cdiv(M, kTile) * cdiv(N, kTile) > (int64_t(1) << 24) || M > (int64_t(1) << 40) / N)
        return FP8MM_ERR_SHAPE;
    if (M == 0)
        return FP8MM_OK;
    if (!A || !B || !sa || !sb || !target)
        return FP8MM_ERR_NULL;
    if ((reinterpret_cast<uintptr_t>(A) & 15) || (reinterpret_cast<uintptr_t>(B) & 15) ||
        (reinterpret_cast<uintptr_t>(sa) & 3) || (reinterpret_cast<uintptr_t>(sb) & 3) ||
        (reinterpret_cast<uintptr_t>(bias) & (row_type_bytes(bias_type) - 1)) || (reinterpret_cast<uintptr_t>(target) & 7))
        return FP8MM_ERR_ALIGN;
    return FP8MM_OK;
}

// Memory of a call: what is written must not overlap anything else of it.
struct Stretch {
    const void *at;
    int64_t bytes;
};
bool overlap(const Stretch &a, const Stretch &b)
{
    const uintptr_t p = reinterpret_cast<uintptr_t>(a.at), q = reinterpret_cast<uintptr_t>(b.at);
    return a.at && b.at && a.bytes > 0 && b.bytes > 0 && p < q + static_cast<uintptr_t>(b.bytes) &&
           q < p + static_cast<uintptr_t>(a.bytes);
}
bool written_apart(std::initializer_list<Stretch> written, std::initializer_list<Stretch> read)
{
    for (const Stretch *w = written.begin(); w != written.end(); ++w) {
        for (const Stretch *o = w + 1; o != written.end(); ++o)
            if (overlap(*w, *o))
                return false;
        for (const Stretch &r : read)
            if (overlap(*w, r))
                return false;
    }
    return true;
}

// A matrix of `rows` x `cols` elements, rows `ld` elements apart, `items` of
// them `item` elements apart, in boxes of box_rows rows x 128 bytes (or 64).
int map_matrix(CUtensorMap *map, CUtensorMapDataType type, int es, const void *base, int64_t rows, int64_t cols, int64_t ld,
               int box_rows, int64_t items = 1, int64_t item = 0, int box_bytes = 128)
{
    const int64_t dims[3] = {cols, rows, items};
    const int64_t strides[2] = {ld * es, (item ? item : ld * rows) * es};
    const int box[3] = {box_bytes / es, box_rows, 1};
    return encode_tiles(map, type, base, dims, strides, box, box_bytes);
}

// The instruction descriptor's operand formats: P gives the rows, Q the columns.
uint32_t formats(int p_type, int q_type)
{
    return (p_type == FP8MM_TYPE_E5M2 ? 1u << 7 : 0u) | (q_type == FP8MM_TYPE_E5M2 ? 1u << 10 : 0u);
}

TileSpace tile_space(int64_t rows, int64_t cols, int width, int64_t kblocks, int splits, int run)
{
    TileSpace t{};
    t.rows = static_cast<int>(rows);
    t.cols = static_cast<int>(cols);
    t.width = width;
    // tiles of equal rows, in whole blocks of 32 per CTA
    t.half = static_cast<int>(cdiv(cdiv(rows, 2 * cdiv(rows, kTile)), 32)) * 32;
    t.kblocks = static_cast<int>(kblocks);
    t.tiles_p = static_cast<int>(cdiv(rows, kTile));
    t.tiles_q = static_cast<int>(cdiv(cols, width));
    t.group = std::min(t.tiles_p, 16);
    t.splits = splits;
    t.run = run;
    t.units_in_group = t.group * static_cast<int>(cdiv(t.tiles_q, run));
    t.num_units = t.tiles_p * static_cast<int>(cdiv(t.tiles_q, run)) * splits;
    return t;
}

template <int KIND>
int launch_tiles(const AllMaps<KIND> &maps, LossParams &p, int sms, cudaStream_t stream)
{
    auto kern = loss_kernel<KIND>;
    using C = Cfg<KIND>;
    static bool attr_set[kMaxDevices] = {};
    int dev = 0;
    cudaGetDevice(&dev);
    if (!attr_set[dev]) {
        const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmemBytes);
        if (e != cudaSuccess)
            return cuda_fail(e, "cudaFuncSetAttribute");
        attr_set[dev] = true;
    }
    const int rc = device_limit(&p.status, &p.timeout_cycles);
    if (rc != FP8MM_OK)
        return rc;
    const int units = p.t[0].num_units + (KIND == kGrad ? p.t[1].num_units : 0);
    return launch_pdl(kern, 2 * std::min(sms / 2, units), C::kThreads, C::kSmemBytes, stream, "cross entropy launch", maps, p);
}

// Tiles of the product z [M, N]: their width, and how many of a row are one unit.
struct TileChoice {
    int width, run;
};

// With many tiles a CTA pair takes several neighbours, over which a row's maximum and
// sum stay in registers and the tile's place is found once: a unit of `run` tiles costs
// about as much as run + 0.2, in turns of 76 pairs. (Not of the device's SMs, so that
// the workspace's size does not depend on them.) 16384 x 8192 x 512: units of 4, 66 us
// (of one tile 71).
int choose_run(int64_t M, int64_t N, int width)
{
    const int64_t rows = cdiv(M, kTile), across = cdiv(N, width);
    int best = 1;
    int64_t cost = INT64_MAX;
    for (int run = 1; run <= 8; run *= 2) {
        const int64_t units = rows * cdiv(across, run), c = cdiv(units, 76) * (5 * run + 1);
        // (fewer leave pairs without any, and some of memory's speed: one row of 32000 columns
        // 30.0 us, in units of two tiles 30.7)
        if (run > 1 && units < 76)
            break;
        if (c < cost) {
            cost = c;
            best = run;
        }
    }
    return best;
}

// The width that ends first, by what a CTA pair loads for its tiles in turn: its
// rows of A (up to 256) and its columns of B (one row of 32000 columns: two turns of
// 224 columns for 256).
TileChoice choose_tiles(int64_t M, int64_t N, int sms)
{
    const int64_t pairs = sms / 2, rows = cdiv(cdiv(M, cdiv(M, kTile)), 64) * 64;
    TileChoice best{kTile, 1};
    int64_t cost = INT64_MAX;
    for (int width = kTile; width >= kLeastWidth; width -= 32) {
        const int64_t c = cdiv(cdiv(M, kTile) * cdiv(N, width), pairs) * (rows + width);
        if (c < cost) {
            cost = c;
            best.width = width;
        }
    }
    best.run = choose_run(M, N, best.width);
    return best;
}

// Parts of a row that kStats leaves, and the most there can be.
int64_t parts_of(const TileChoice &t, int64_t N) { return cdiv(cdiv(N, t.width), t.run) * 4; }
int64_t most_parts(int64_t M, int64_t N)
{
    int64_t most = 0;
    for (int width = kLeastWidth; width <= kTile; width += 32)
        most = std::max(most, parts_of({width, choose_run(M, N, width)}, N));
    return most;
}

// The operands' maps and the tile space of z [M, N] (kStats, kSlope).
int product_maps(const TileChoice &t, const void *A, int a_type, const void *B, int b_type, int64_t M, int64_t N, int64_t K,
                 Maps &m, LossParams &p)
{
    constexpr CUtensorMapDataType u8 = CU_TENSOR_MAP_DATA_TYPE_UINT8;
    p.t[0] = tile_space(M, N, t.width, cdiv(K, 128), 1, t.run);
    p.t[0].idesc = fp8mm::ptx::idesc_e4m3_f32(kTile, t.width) | formats(a_type, b_type);
    p.M = static_cast<int>(M);
    p.N = static_cast<int>(N);
    const int rc = map_matrix(&m.a, u8, 1, A, M, K, K, p.t[0].half);
    return rc != FP8MM_OK ? rc : map_matrix(&m.b, u8, 1, B, N, K, K, t.width / 2);
}

// K slices of the gradients' products, which share one launch: tiles ta of ka blocks
// of 64, tb of kb (0 tiles: not wanted). Chosen by when the last CTA pair ends: a block takes
// a pair 0.28 us, a tile's end 1.5; sums of slices are written as fp32 partials and
// read by another kernel (2 us and 5.5 TB/s). 2048 x 2048 x 512, 16 tiles each:
// two slices each, one turn of 64 units (chosen apart: four each, two turns).
struct Slices {
    int a, b;
};
Slices choose_slices(int64_t ta, int64_t ka, int64_t out_a, int64_t tb, int64_t kb, int64_t out_b, int sms)
{
    constexpr int kCounts[] = {1, 2, 3, 4, 5, 6, 8, 10, 12, 16, 19, 24, 32, 38, 48, 64};
    const int64_t pairs = sms / 2;
    auto unit = [](int64_t blocks, int slices) { return cdiv(blocks, slices) * 0.28 + 1.5; };
    auto sums = [](int64_t out, int slices) { return slices > 1 ? 2.0 + static_cast<double>(out) * slices * 8 / 5.5e6 : 0.0; };
    Slices best{1, 1};
    double least = 0.0;
    for (int sa : kCounts) {
        if (sa > 1 && (ta == 0 || sa * 4 > ka))
            break;
        for (int sb : kCounts) {
            if (sb > 1 && (tb == 0 || sb * 4 > kb))
                break;
            // unit u goes to pair u % pairs, A's first: the pair with the most is the first
            // one, or the first without A's odd unit
            const int64_t ua = ta * sa, u = ua + tb * sb;
            double t = 0.0;
            for (int64_t p : {int64_t(0), ua % pairs}) {
                const int64_t na = cdiv(std::max<int64_t>(ua - p, 0), pairs), n = cdiv(std::max<int64_t>(u - p, 0), pairs);
                t = std::max(t, static_cast<double>(na) * unit(ka, sa) + static_cast<double>(n - na) * unit(kb, sb));
            }
            t += sums(out_a, sa) + sums(out_b, sb);
            if ((sa == 1 && sb == 1) || t < least) {
                least = t;
                best = {sa, sb};
            }
        }
    }
    return best;
}

// How a gradient call goes through the vocabulary, and where its workspace's
// parts are.
struct GradPlan {
    int64_t piece, pieces;                       // columns of a piece (a multiple of 256, or all), how many
    int split_a, split_b;
    bool parts_a, parts_b;                       // results pass through fp32 partials
    int64_t norms, h16, w16, dz, colsum, parts_a_at, parts_b_at, bytes;
};

GradPlan plan_grad(int64_t M, int64_t N, int64_t K, bool da, bool db, bool dbias, int sms)
{
    GradPlan g{};
    const int64_t most = std::max<int64_t>(kTile, kPieceBytes / 2 / std::max(M, K) / kTile * kTile);
    g.pieces = cdiv(N, most);
    g.piece = cdiv(cdiv(N, g.pieces), kTile) * kTile;
    g.pieces = cdiv(N, g.piece);
    const int64_t n = std::min(N, g.piece), across = cdiv(K, kTile);
    const Slices s = choose_slices(da ? cdiv(M, kTile) * across : 0, cdiv(n, 64), M * K, db ? cdiv(n, kTile) * across : 0, cdiv(M, 64),
                                   n * K, sms);
    g.split_a = s.a;
    g.split_b = s.b;
    g.parts_a = da && (g.split_a > 1 || g.pieces > 1);
    g.parts_b = db && g.split_b > 1;
    int64_t at = 0;
    auto take = [&](int64_t bytes) {
        const int64_t here = at;
        at += aligned(bytes);
        return here;
    };
    g.norms = take(3 * kNormParts * 4);
    g.dz = take(M * g.piece * 2);
    g.h16 = take(db ? M * K * 2 : 0);
    g.w16 = take(da ? g.piece * K * 2 : 0);
    g.colsum = take(dbias ? cdiv(M, 32) * g.piece * 4 : 0);
    g.parts_a_at = take(g.parts_a ? g.split_a * M * K * 4 : 0);
    g.parts_b_at = take(g.parts_b ? g.split_b * g.piece * K * 4 : 0);
    g.bytes = at;
    return g;
}

int64_t stats_bytes(int64_t M, int64_t N) { return aligned(most_parts(M, N) * M * 8); }

int zero(void *p, int64_t bytes, cudaStream_t s)
{
    const cudaError_t e = p ? cudaMemsetAsync(p, 0, static_cast<size_t>(bytes), s) : cudaSuccess;
    return e == cudaSuccess ? FP8MM_OK : cuda_fail(e, "cudaMemsetAsync(gradient)");
}

int finish(const void *parts, int64_t n, int count, int out_type, int norm_of, const uint32_t *norms, float factor,
           void *out, int sms, cudaStream_t s)
{
    FinishParams f{};
    f.parts = static_cast<const float *>(parts);
    f.n = n;
    f.count = count;
    f.out_type = out_type;
    f.norm_of = norm_of;
    f.norms = norms;
    f.factor = factor;
    f.out = out;
    // (where whole CTAs of elements are less than two turns of the SMs' eight)
    const int64_t most = static_cast<int64_t>(sms) * 8;
    if (count >= 8 && n / 4 < 2 * most * kFinishThreads)
        return launch_grid2(finish_kernel<8>, std::min<int64_t>(cdiv(n / 4, kFinishThreads / 8), most), 1, kFinishThreads, s,
                            "gradient sum launch", f);
    return launch_grid2(finish_kernel<1>, std::min<int64_t>(cdiv(n / 4, kFinishThreads), most), 1, kFinishThreads, s,
                        "gradient sum launch", f);
}

constexpr CUtensorMapDataType kF16 = CU_TENSOR_MAP_DATA_TYPE_FLOAT16,
                              kF32 = CU_TENSOR_MAP_DATA_TYPE_FLOAT32, kB16 = CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;

}  // namespace

extern "C" {

int64_t fp8_cross_entropy_workspace(int64_t M, int64_t N)
{
    if (M < 0 || N < 1 || M > kMostRows || N > kMostRows || M > (int64_t(1) << 40) / N)
        return FP8MM_ERR_SHAPE;
    return M == 0 ? 0 : stats_bytes(M, N) + aligned(M * 4);
}

int fp8_cross_entropy(const void *A, int a_type, const void *B, int b_type, const float *scale_a, const float *scale_b,
                      int scale_mode, const void *bias, int bias_type, const int64_t *target, int64_t ignore_index,
                      float *loss, float *lse, int64_t M, int64_t N, int64_t K, void *workspace, int64_t workspace_bytes,
                      void *stream)
{
    int rc = check_problem(A, B, scale_a, scale_b, scale_mode, a_type, b_type, bias, bias_type, target, M, N, K);
    if (rc != FP8MM_OK || M == 0)
        return rc;
    if (!loss || !lse || !workspace)
        return FP8MM_ERR_NULL;
    if ((reinterpret_cast<uintptr_t>(loss) & 3) || (reinterpret_cast<uintptr_t>(lse) & 3) ||
        (reinterpret_cast<uintptr_t>(workspace) & 15))
        return FP8MM_ERR_ALIGN;
    const int64_t need = fp8_cross_entropy_workspace(M, N), scales = scale_mode == FP8MM_SCALE_ROWWISE ? 4 : 0;
    if (workspace_bytes < need)
        return FP8MM_ERR_SHAPE;
    if (!written_apart({{loss, M * 4}, {lse, M * 4}, {workspace, need}},
                       {{A, M * K}, {B, N * K}, {scale_a, std::max<int64_t>(4, scales * M)}, {scale_b, std::max<int64_t>(4, scales * N)},
                        {bias, N * row_type_bytes(bias_type)}, {target, M * 8}}))
        return FP8MM_ERR_MODE;
    int sms = 0;
    if ((rc = device_sms(&sms)) != FP8MM_OK)
        return rc;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const TileChoice t = choose_tiles(M, N, sms);
    LossParams p{};
    AllMaps<kStats> maps{};
    if ((rc = product_maps(t, A, a_type, B, b_type, M, N, K, maps.of[0], p)) != FP8MM_OK)
        return rc;
    p.scale_a = scale_a;
    p.scale_b = scale_b;
    p.rowwise = scale_mode == FP8MM_SCALE_ROWWISE;
    p.bias = bias;
    p.bias_type = bias_type;
    p.target = target;
    p.ignore = ignore_index;
    p.vocabulary = N;
    p.stats = static_cast<float2 *>(workspace);
    p.target_z = reinterpret_cast<float *>(static_cast<uint8_t *>(workspace) + stats_bytes(M, N));
    if ((rc = launch_tiles<kStats>(maps, p, sms, s)) != FP8MM_OK)
        return rc;
    CombineParams c{};
    c.stats = p.stats;
    c.target_z = p.target_z;
    c.target = target;
    c.ignore = ignore_index;
    c.vocabulary = N;
    c.loss = loss;
    c.lse = lse;
    c.rows = static_cast<int>(M);
    c.parts = static_cast<int>(parts_of(t, N));
    // (up to where the rows' CTAs are a few on every SM, and a sector's other rows are not
    // read again too often)
    if (M <= 4 * sms)
        return launch_grid2(combine_row_kernel, M, 1, kRowThreads, s, "cross entropy sum launch", c);
    return launch_grid2(combine_kernel, cdiv(M, 32), 1, kCombineThreads, s, "cross entropy sum launch", c);
}

int64_t fp8_cross_entropy_grad_workspace(int64_t M, int64_t N, int64_t K, int want_da, int want_db, int want_dbias)
{
    if (M < 0 || N < 1 || M > kMostRows || N > kMostRows || K < 16 || K % 16 != 0 || K > (int64_t(1) << 24) ||
        cdiv(M, kTile) * cdiv(N, kTile) > (int64_t(1) << 24) || M > (int64_t(1) << 40) / N)
        return FP8MM_ERR_SHAPE;
    if (M == 0 || !(want_da || want_db || want_dbias))
        return 0;
    int sms = 0;
    const int rc = device_sms(&sms);
    if (rc != FP8MM_OK)
        return rc;
    return plan_grad(M, N, K, want_da != 0, want_db != 0, want_dbias != 0, sms).bytes;
}

int fp8_cross_entropy_grad(const void *A, int a_type, const void *B, int b_type, const float *scale_a,
                           const float *scale_b, int scale_mode, const void *bias, int bias_type, const int64_t *target,
                           int64_t ignore_index, const float *lse, const float *dloss, int64_t dloss_count, void *da,
                           void *db, int out_type, float *dbias, int64_t M, int64_t N, int64_t K, void *workspace,
                           int64_t workspace_bytes, void *stream)
{
    int rc = check_problem(A, B, scale_a, scale_b, scale_mode, a_type, b_type, bias, bias_type, target, M, N, K);
    if (rc != FP8MM_OK)
        return rc;
    if (!row_type_known(out_type))
        return FP8MM_ERR_MODE;
    if (dloss_count != 1 && dloss_count != M)
        return FP8MM_ERR_SHAPE;
    if ((reinterpret_cast<uintptr_t>(lse) & 3) || (reinterpret_cast<uintptr_t>(dloss) & 3) ||
        (reinterpret_cast<uintptr_t>(dbias) & 3) || (reinterpret_cast<uintptr_t>(da) & 15) ||
        (reinterpret_cast<uintptr_t>(db) & 15) || (reinterpret_cast<uintptr_t>(workspace) & 15))
        return FP8MM_ERR_ALIGN;
    if (!da && !db && !dbias)
        return FP8MM_OK;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    int sms = 0;
    const int es = static_cast<int>(row_type_bytes(out_type));
    const int64_t scales = scale_mode == FP8MM_SCALE_ROWWISE ? 4 : 0;
    const std::initializer_list<Stretch> inputs = {
        {A, M * K}, {B, N * K}, {scale_a, std::max<int64_t>(4, scales * M)}, {scale_b, std::max<int64_t>(4, scales * N)},
        {bias, N * row_type_bytes(bias_type)}, {target, M * 8}, {lse, M * 4}, {dloss, dloss_count * 4}};
    const std::initializer_list<Stretch> outputs = {{da, M * K * es}, {db, N * K * es}, {dbias, N * 4}};
    if (!written_apart(outputs, inputs) || !written_apart(outputs, {{workspace, workspace_bytes}}))
        return FP8MM_ERR_MODE;
    if (M == 0) {
        // sums over no rows
        if ((rc = device_sms(&sms)) != FP8MM_OK || (rc = zero(db, N * K * es, s)) != FP8MM_OK)
            return rc;
        return zero(dbias, N * 4, s);
    }
    if (!lse || !dloss || !workspace)
        return FP8MM_ERR_NULL;
    if ((rc = device_sms(&sms)) != FP8MM_OK)
        return rc;
    const GradPlan g = plan_grad(M, N, K, da != nullptr, db != nullptr, dbias != nullptr, sms);
    if (workspace_bytes < g.bytes)
        return FP8MM_ERR_SHAPE;
    if (!written_apart({{workspace, g.bytes}}, inputs))
        return FP8MM_ERR_MODE;
    uint8_t *ws = static_cast<uint8_t *>(workspace);
    uint32_t *norms = reinterpret_cast<uint32_t *>(ws + g.norms);
    const int rowwise = scale_mode == FP8MM_SCALE_ROWWISE;
    const CUtensorMapDataType out_map = out_type == FP8MM_OUT_F32 ? kF32 : out_type == FP8MM_OUT_F16 ? kF16 : kB16;
    // what comes off dz W16 and dz^T H16 beside the norms
    const float factor_a = 1.0f / (kSlopeScale * code_scale(b_type)), factor_b = 1.0f / (kSlopeScale * code_scale(a_type));

    // Few values' norms are found by each CTA of the first piece itself, beside its first
    // loads: a launch less (128 x 4096 x 480 18.3 to 17.2 us).
    const bool few = M <= kFewNorms && N <= kFewNorms && g.pieces == 1;
    NormsParams n{};
    n.dloss = dloss;
    n.dloss_step = dloss_count == 1 ? 0 : 1;
    n.rowwise = rowwise;
    n.scale_b = scale_b;
    n.scale_a = scale_a;
    n.target = target;
    n.ignore = ignore_index;
    n.count[kNormG] = M;
    n.count[kNormB] = rowwise ? N : 1;
    n.count[kNormH] = M;
    n.out = norms;
    if (!few && (rc = launch_grid2(norms_kernel, kNormParts, 3, kNormThreads, s, "cross entropy norms launch", n)) != FP8MM_OK)
        return rc;

    for (int64_t i = 0; i < g.pieces; ++i) {
        const int64_t n0 = i * g.piece, nv = std::min(g.piece, N - n0);
        const uint8_t *Bi = static_cast<const uint8_t *>(B) + n0 * K;
        const float *sbi = scale_b + (rowwise ? n0 : 0);
        LossParams p{};
        AllMaps<kSlope> maps{};
        if ((rc = product_maps(choose_tiles(M, nv, sms), A, a_type, Bi, b_type, M, nv, K, maps.of[0], p)) != FP8MM_OK)
            return rc;
        p.scale_a = scale_a;
        p.scale_b = sbi;
        p.rowwise = rowwise;
        p.bias = bias ? static_cast<const uint8_t *>(bias) + n0 * row_type_bytes(bias_type) : nullptr;
        p.bias_type = bias_type;
        p.target = target;
        p.ignore = ignore_index;
        p.col0 = n0;
        p.vocabulary = N;
        p.lse = lse;
        p.dloss = dloss;
        p.dloss_step = n.dloss_step;
        p.colsum = dbias ? reinterpret_cast<float *>(ws + g.colsum) : nullptr;
        p.colsum_ld = g.piece;
        p.norms = norms;
        p.norms_out = few ? norms : nullptr;
        p.w16 = da ? reinterpret_cast<__half *>(ws + g.w16) : nullptr;
        p.h16 = db && i == 0 ? reinterpret_cast<__half *>(ws + g.h16) : nullptr;
        p.K = static_cast<int>(K);
        p.a_type = a_type;
        p.b_type = b_type;
        // dz [M, nv] with rows of `piece` elements, written in blocks of 32 x 32
        if ((rc = map_matrix(&maps.of[0].out, kF16, 2, ws + g.dz, M, nv, g.piece, 32, 1, 0, 64)) != FP8MM_OK ||
            (rc = launch_tiles<kSlope>(maps, p, sms, s)) != FP8MM_OK)
            return rc;
        if (dbias) {
            ColumnsParams c{};
            c.parts = p.colsum;
            c.ld = g.piece;
            c.cols = static_cast<int>(nv);
            c.count = static_cast<int>(cdiv(M, 32));
            c.norms = norms;
            c.out = dbias + n0;
            if ((rc = launch_grid2(columns_kernel, cdiv(nv, 32), 1, kColumnsThreads, s, "bias gradient sum launch", c)) != FP8MM_OK)
                return rc;
        }
        if (!da && !db)
            continue;
        LossParams o{};
        AllMaps<kGrad> to{};
        o.rowwise = rowwise;
        o.norms = norms;
        o.target = target;
        o.ignore = ignore_index;
        o.dloss = dloss;
        o.dloss_step = n.dloss_step;
        if (da) {
            // (a last piece with fewer blocks than slices adds to the first partials only)
            TileSpace &t = o.t[kOfA];
            t = tile_space(M, K, kTile, cdiv(nv, 64), static_cast<int>(std::min<int64_t>(g.split_a, cdiv(nv, 64))), 1);
            t.idesc = fp8mm::ptx::idesc_f16_f32(kTile, kTile, false, true);
            Maps &m = to.of[kOfA];
            if ((rc = map_matrix(&m.a, kF16, 2, ws + g.dz, M, nv, g.piece, t.half)) != FP8MM_OK ||
                (rc = map_matrix(&m.b, kF16, 2, ws + g.w16, nv, K, K, 64)) != FP8MM_OK ||
                (rc = g.parts_a ? map_matrix(&m.out, kF32, 4, ws + g.parts_a_at, M, K, K, 32, g.split_a)
                                : map_matrix(&m.out, out_map, es, da, M, K, K, 32)) != FP8MM_OK)
                return rc;
            o.r[kOfA] = {!g.parts_a, factor_a, kNormB, scale_a, g.parts_a ? FP8MM_OUT_F32 : out_type, i > 0};
        }
        uint8_t *dbi = db ? static_cast<uint8_t *>(db) + n0 * K * es : nullptr;
        if (db) {
            TileSpace &t = o.t[kOfB];
            t = tile_space(nv, K, kTile, cdiv(M, 64), g.split_b, 1);
            t.half = 128;              // (MN-major rows come in boxes of 64)
            t.idesc = fp8mm::ptx::idesc_f16_f32(kTile, kTile, true, true);
            Maps &m = to.of[kOfB];
            if ((rc = map_matrix(&m.a, kF16, 2, ws + g.dz, M, nv, g.piece, 64)) != FP8MM_OK ||
                (rc = map_matrix(&m.b, kF16, 2, ws + g.h16, M, K, K, 64)) != FP8MM_OK ||
                (rc = g.parts_b ? map_matrix(&m.out, kF32, 4, ws + g.parts_b_at, nv, K, K, 32, g.split_b)
                                : map_matrix(&m.out, out_map, es, dbi, nv, K, K, 32)) != FP8MM_OK)
                return rc;
            o.r[kOfB] = {!g.parts_b, factor_b, kNormH, sbi, g.parts_b ? FP8MM_OUT_F32 : out_type, 0};
        }
        // (the maps of a product that is not wanted have no tiles)
        if (!da)
            to.of[kOfA] = to.of[kOfB];
        if (!db)
            to.of[kOfB] = to.of[kOfA];
        if ((rc = launch_tiles<kGrad>(to, o, sms, s)) != FP8MM_OK)
            return rc;
        if (g.parts_b && (rc = finish(ws + g.parts_b_at, nv * K, g.split_b, out_type, kNormH, norms, factor_b, dbi, sms, s)) != FP8MM_OK)
            return rc;
    }
    if (g.parts_a)
        return finish(ws + g.parts_a_at, M * K, g.split_a, out_type, kNormB, norms, factor_a, da, sms, s);
    return FP8MM_OK;
}

}  // extern "C"
