// Gated block, bf16.
#include "prod_api.hpp"
#include "prod_launch.hpp"

template <>
hipError_t tg::launch_glu<1>(const ProdArgs &p, const GluEpi<1> &e, hipStream_t s) {
    return launch_prod<1, true>(p, e, s);
}
