// Cross attention: which kernels a call runs, and its workspace.
#include "attention.cuh"

namespace gs {

namespace {

size_t round256(size_t n) { return (n + 255) / 256 * 256; }

size_t delta_bytes(const AttnArgs& a) { return round256((size_t)a.batch * a.heads * a.len_q * sizeof(float)); }

}  // namespace

size_t attn_workspace_bytes(const AttnArgs& a, bool backward) { return backward ? delta_bytes(a) : 0; }

cudaError_t launch_attn_fwd(const AttnArgs& a, void* workspace, cudaStream_t st) { return launch_attn_simt(a, false, st); }

cudaError_t launch_attn_bwd(const AttnArgs& args, void* workspace, cudaStream_t st) {
    AttnArgs a = args;
    a.delta = static_cast<float*>(workspace);
    cudaError_t e = launch_attn_delta(a, st);
    return e ? e : launch_attn_simt(a, true, st);
}

}  // namespace gs
