// What the translation units behind include/relation.h share on the host.
#pragma once

#include "../../include/relation.h"
#include "kernels.h"

namespace relation {

// The current device's status word and SM count.
relation_status_t api_device(unsigned int** status, int* num_sms);

// Sets what relation_last_launch_count() returns on this thread.
void api_set_launches(int n);

// RoPE frequencies base^(-2c/d) / (2 pi), c < d/2 (base <= 0: disabled).
RopeTable rope_table(int d, float base);

}  // namespace relation
