// sdpa_cache.cu -- C ABI of the calls around the paged cache, the norm and the
// rotation (declared in include/sdpa.h).
#include "cache_api.cuh"

namespace sdpa_host {

cudaError_t take_cache_error(unsigned int* code)
{
    return take_error_word(code);
}

}  // namespace sdpa_host
