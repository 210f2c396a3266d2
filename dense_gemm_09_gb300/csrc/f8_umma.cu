#include "f8.cuh"
namespace dgemm {
bool f8_umma_config_ok(const F8Config &) { return false; }
bool launch_f8_umma(const F8Params &, const F8Config &, cudaStream_t) { return false; }
}
