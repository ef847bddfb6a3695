// santa_diff_chunk.cu -- differential heads, many query rows: launches of the kernel
// in santa_chunk.cuh, all of whose sums go through memory.
#include "santa_chunk.cuh"

namespace santa {

namespace {

template <typename T, bool E4M3, int D>
cudaError_t inst(const JoinArgs& a, bool behind) {
  using Gm = ChunkGeom<E4M3, D, diff_columns<E4M3, D, true>(), true>;
  auto kern = paged_chunk_kernel<T, E4M3, D, JoinArgs, true>;
  static std::atomic<unsigned long long> raised{0};
  const cudaError_t e = raise_smem((const void*)kern, (int)Gm::SMEM, raised);
  if (e != cudaSuccess) return e;
  CUtensorMap tq, tk, tv;
  if (!encode_pairs(&tq, a.q, D, a.H, a.total_q, a.G, TROWS / a.G) || !encode_cache<E4M3, D>(&tk, a, a.K) ||
      !encode_cache<E4M3, D>(&tv, a, a.V))
    return cudaErrorInvalidValue;
  return launch_pass(kern, (unsigned)a.splits, Gm::THREADS, Gm::SMEM, a.stream, behind, tq, tk, tv, a);
}
template <typename T>
cudaError_t type(const JoinArgs& a, bool behind) {
  if (a.D == 128) return inst<T, true, 128>(a, behind);   // over 16 bits: santa_diff_wide.cu
  return a.e4m3 ? inst<T, true, 64>(a, behind) : inst<T, false, 64>(a, behind);
}

}  // namespace

cudaError_t launch_diff_chunk(const JoinArgs& a, bool behind) {
  return a.dtype == 0 ? type<bf16_t>(a, behind) : type<fp16_t>(a, behind);
}

}  // namespace santa
