#include "paged_sched.cuh"
namespace ds4g {
bool paged_attn_tc_ok(const PagedKV &, int, int, int) { return false; }
int paged_attn_tc_rows(int group, int max_new) { return 128 / group * group; }
cudaError_t paged_attn_tc(const AttnArgs &, cudaStream_t, int) { return cudaErrorNotSupported; }
}
