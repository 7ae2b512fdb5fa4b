// paged_bf16.cu -- attention over the paged cache for bf16 queries.
#include "paged_launch.cuh"

template vattn_status vattn::host::paged_dispatch<__nv_bfloat16>(const PagedParams&, const Pools&, int, int, cudaStream_t);
