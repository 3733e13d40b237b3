// fp8mm_adamw.cu -- C entry of the AdamW step over many tensors.
#include "fp8mm_adamw.cuh"
#include "fp8mm_rows_host.h"

#include <cmath>
#include <exception>
#include <vector>

namespace {

using namespace fp8mm_host;
using namespace fp8adam;

bool aligned_to(const void *p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

// A stretch of memory that a call writes, or reads only.
struct Stretch {
    uintptr_t from, to;
    bool written;
};

// The stretches in order of their beginnings. Tensors mostly lie in memory in the order of
// their list, and a list for each role is a run that ascends: a few runs are merged, more
// (tensors in any order) sorted. 336 stretches, on the host: 0.4 us merged from 7 runs, 3 us
// sorted; in random order 17 us sorted, 27 us merged.
void ascend(std::vector<Stretch> &all, std::vector<Stretch> &other, std::vector<size_t> &runs)
{
    auto before = [](const Stretch &a, const Stretch &b) { return a.from < b.from; };
    for (;;) {
        runs.clear();
        for (size_t i = 0; i < all.size(); ++i)
            if (i == 0 || before(all[i], all[i - 1]))
                runs.push_back(i);
        if (runs.size() <= 1)
            return;
        if (runs.size() > 16) {
            std::sort(all.begin(), all.end(), before);
            return;
        }
        runs.push_back(all.size());
        other.resize(all.size());
        const size_t last = runs.size() - 1;
        for (size_t r = 0; r < last; r += 2) {
            const size_t middle = runs[r + 1], end = r + 2 <= last ? runs[r + 2] : middle;
            std::merge(all.begin() + runs[r], all.begin() + middle, all.begin() + middle, all.begin() + end,
                       other.begin() + runs[r], before);
        }
        all.swap(other);
    }
}

template <int BITS, bool W32, bool MASTER, bool G32, int T>
int launch(const Params<T> &p, int sms, cudaStream_t stream)
{
    // as many CTAs as run at once, a block of 256 elements a warp and turn
    const int64_t grid = std::min<int64_t>(cdiv(p.blocks, kThreads / 32), static_cast<int64_t>(sms) * kCtasPerSm);
    return launch_pdl(adamw_kernel<BITS, W32, MASTER, G32, T>, static_cast<int>(grid), kThreads, 0, stream, "AdamW launch", p);
}

template <int BITS, bool G32, int T>
int launch_types(const Params<T> &p, bool masters, int sms, cudaStream_t stream)
{
    if (masters)
        return launch<BITS, true, true, G32>(p, sms, stream);
    return p.param_type == FP8MM_OUT_F32 ? launch<BITS, true, false, G32>(p, sms, stream)
                                         : launch<BITS, false, false, G32>(p, sms, stream);
}

// Tensors [from, to) of the call, T at most, which hold anything.
template <int T>
int step_some(const fp8mm_adamw_tensor *tensors, int64_t from, int64_t to, const fp8mm_adamw_options &o, int bits, const Hyper &h,
              int sms, cudaStream_t stream)
{
    Params<T> p{};
    p.h = h;
    p.param_type = o.param_type;
    p.grad_type = o.grad_type;
    bool masters = false;              // (all have one, or none)
    const int code = bits == 8 ? 8 : 16;              // alignment of 8 elements of a state
    for (int64_t i = from; i < to; ++i) {
        const fp8mm_adamw_tensor &a = tensors[i];
        if (a.count == 0)
            continue;
        p.first[p.tensors] = p.blocks;
        Tensor &t = p.t[p.tensors++];
        t.param = a.param;
        t.grad = a.grad;
        t.master = a.master;
        t.m = a.exp_avg;
        t.v = a.exp_avg_sq;
        t.m_scale = a.exp_avg_scale;
        t.v_scale = a.exp_avg_sq_scale;
        t.count = a.count;
        t.vec = aligned_to(a.param, 16) && aligned_to(a.grad, 16) && aligned_to(a.master, 16) && aligned_to(t.m, code) &&
                aligned_to(t.v, code);
        masters = a.master != nullptr;
        p.blocks += cdiv(a.count, kBlock);
    }
    if (p.tensors == 0)
        return FP8MM_OK;
    if (p.grad_type == FP8MM_OUT_F32)
        return bits == 8 ? launch_types<8, true>(p, masters, sms, stream) : launch_types<32, true>(p, masters, sms, stream);
    return bits == 8 ? launch_types<8, false>(p, masters, sms, stream) : launch_types<32, false>(p, masters, sms, stream);
}

}  // namespace

extern "C" int fp8_adamw(const fp8mm_adamw_tensor *tensors, int64_t n, const fp8mm_adamw_options *options, void *stream)
{
    if (!options || (n > 0 && !tensors))
        return FP8MM_ERR_NULL;
    const fp8mm_adamw_options &o = *options;
    const bool stochastic = o.state_bits == (8 | FP8MM_STOCHASTIC_EXP_AVG);
    const int bits = stochastic ? 8 : o.state_bits;
    if (!row_type_known(o.param_type) || !row_type_known(o.grad_type) || (bits != 8 && bits != 32))
        return FP8MM_ERR_MODE;
    if (n < 0 || n > (int64_t(1) << 32) || (!o.step_device && o.step < 1) || !std::isfinite(o.lr) || !(o.beta1 >= 0.0 && o.beta1 < 1.0) ||
        !(o.beta2 >= 0.0 && o.beta2 < 1.0) || !(o.eps >= 0.0 && std::isfinite(o.eps)) || !std::isfinite(o.weight_decay))
        return FP8MM_ERR_SHAPE;
    if (!aligned_to(o.lr_device, 4) || !aligned_to(o.step_device, 8) || !aligned_to(o.grad_scale, 4))
        return FP8MM_ERR_ALIGN;
    const int64_t param_bytes = row_type_bytes(o.param_type), grad_bytes = row_type_bytes(o.grad_type);
    const int64_t state_bytes = bits / 8;
    std::vector<Stretch> all, other;
    std::vector<size_t> runs;
    try {
        const size_t most = static_cast<size_t>(n) * 7 + 3;
        all.reserve(most);
        other.reserve(most);
        runs.reserve(most + 1);
    } catch (const std::exception &) {
        set_error("fp8_adamw: no host memory for the check of the tensors");
        return FP8MM_ERR_CUDA;
    }
    auto note = [&](const void *p, int64_t bytes, bool written) {
        const uintptr_t at = reinterpret_cast<uintptr_t>(p);
        if (p)
            all.push_back({at, at + static_cast<uintptr_t>(bytes), written});
    };
    const bool masters = n > 0 && tensors[0].master;
    bool any = false;
    for (int64_t i = 0; i < n; ++i) {
        const fp8mm_adamw_tensor &t = tensors[i];
        if (t.count < 0 || t.count > (int64_t(1) << 40))
            return FP8MM_ERR_SHAPE;
        if ((t.master != nullptr) != masters)
            return FP8MM_ERR_MODE;
        if (t.count == 0)
            continue;
        if (!t.param || !t.grad || !t.exp_avg || !t.exp_avg_sq ||
            (bits == 8 && (!t.exp_avg_scale || !t.exp_avg_sq_scale)))
            return FP8MM_ERR_NULL;
        if (!aligned_to(t.param, param_bytes) || !aligned_to(t.grad, grad_bytes) || !aligned_to(t.master, 4) ||
            !aligned_to(t.exp_avg, state_bytes) || !aligned_to(t.exp_avg_sq, state_bytes) ||
            (bits == 8 && (!aligned_to(t.exp_avg_scale, 4) || !aligned_to(t.exp_avg_sq_scale, 4))))
            return FP8MM_ERR_ALIGN;
        any = true;
    }
    if (!any)
        return FP8MM_OK;
    auto note_all = [&](auto pointer, int64_t bytes, int64_t elements, bool written) {
        for (int64_t i = 0; i < n; ++i)
            if (tensors[i].count > 0)
                note(tensors[i].*pointer, cdiv(tensors[i].count, elements) * bytes, written);
    };
    using T = fp8mm_adamw_tensor;
    note_all(&T::param, param_bytes, 1, true);
    note_all(&T::grad, grad_bytes, 1, false);
    note_all(&T::master, 4, 1, true);
    note_all(&T::exp_avg, state_bytes, 1, true);
    note_all(&T::exp_avg_sq, state_bytes, 1, true);
    if (bits == 8) {
        note_all(&T::exp_avg_scale, 4, kBlock, true);
        note_all(&T::exp_avg_sq_scale, 4, kBlock, true);
    }
    // (read when the CTAs begin, some after others have written)
    note(o.lr_device, 4, false);
    note(o.step_device, 8, false);
    note(o.grad_scale, 4, false);
    // what is written belongs to one tensor: a tensor given twice would be updated
    // by two warps at once
    ascend(all, other, runs);
    uintptr_t end = 0, written_end = 0;
    for (const Stretch &s : all) {
        if (s.from < (s.written ? end : written_end)) {
            set_error("fp8_adamw: two of the tensors share memory that is written");
            return FP8MM_ERR_MODE;
        }
        end = std::max(end, s.to);
        if (s.written)
            written_end = std::max(written_end, s.to);
    }
    int sms = 0;
    int rc = device_sms(&sms);
    if (rc != FP8MM_OK)
        return rc;
    Hyper h{};
    const double rest1 = o.step_device ? 1.0 : 1.0 - std::pow(o.beta1, static_cast<double>(o.step));
    const double rest2 = o.step_device ? 1.0 : 1.0 - std::pow(o.beta2, static_cast<double>(o.step));
    h.keep = static_cast<float>(1.0 - o.lr * o.weight_decay);
    h.b1 = static_cast<float>(o.beta1);
    h.b1c = static_cast<float>(1.0 - o.beta1);
    h.b2 = static_cast<float>(o.beta2);
    h.b2c = static_cast<float>(1.0 - o.beta2);
    h.eps = static_cast<float>(o.eps);
    h.step_size = static_cast<float>(o.lr / rest1);
    h.root = static_cast<float>(1.0 / std::sqrt(rest2));
    h.lr = o.lr;
    h.rest1 = rest1;
    h.beta1 = o.beta1;
    h.beta2 = o.beta2;
    h.weight_decay = o.weight_decay;
    h.lr_device = o.lr_device;
    h.step_device = o.step_device;
    h.step = static_cast<uint32_t>(o.step);
    h.stochastic = stochastic;
    h.grad_scale = o.grad_scale;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (n <= kFew)
        return step_some<kFew>(tensors, 0, n, o, bits, h, sms, s);
    if (n <= kSome)
        return step_some<kSome>(tensors, 0, n, o, bits, h, sms, s);
    for (int64_t i = 0; i < n; i += kMany)
        if ((rc = step_some<kMany>(tensors, i, std::min<int64_t>(n, i + kMany), o, bits, h, sms, s)) != FP8MM_OK)
            return rc;
    return FP8MM_OK;
}
