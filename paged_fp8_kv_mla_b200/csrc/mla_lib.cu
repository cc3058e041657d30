// The library's one translation unit: the decode's C ABI and the cache operators' C ABI, which share
// the error text, the device status word and the host helpers.
#include "mla_api.cu"
#include "mla_cache_api.cuh"
