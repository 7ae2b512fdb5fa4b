// paged_f16.cu -- attention over the paged cache for f16 queries.
#include "paged_launch.cuh"

template vattn_status vattn::host::paged_dispatch<__half>(const PagedParams&, const Pools&, int, int, cudaStream_t);
