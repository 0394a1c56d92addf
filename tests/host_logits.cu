// host_logits.cu -- prints how qmm_logits_adjust cuts its rows, on the host:
// arguments SMs, then triples of rows, vocabulary and bytes of a logit; a line
// of parts, logits of a part, and tokens counted at once for each.
#include <cstdio>
#include <cstdlib>

#include "../quantized_gguf_dequant_gb300/csrc/qmm_internal.h"

int main(int argc, char **argv)
{
    for (int i = 2; i + 2 < argc; i += 3) {
        const qmm::LogitsPlan p =
            qmm::plan_logits(atoll(argv[i]), atoll(argv[i + 1]), atoi(argv[i + 2]), atoi(argv[1]));
        printf("%d %d %d\n", p.parts, p.part, p.at_once);
    }
    return 0;
}
