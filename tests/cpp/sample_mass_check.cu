// The samplers' fixed-point scale on the host: the masses of every vocabulary
// they accept (and of wider ones, for models) add up within 64 bits.
#include <cstdio>

#include "../../decoder_only_transformer_llama_b200/csrc/sample_mass.cuh"

#define CHECK(x) do { if (!(x)) { printf("V=%d: %s\n", V, #x); return 1; } } while (0)

int main() {
    for (int V = 1; V > 0 && V <= 0x7fffffff - 3; V = V < 600000 ? V + 1 : (V < 0x3fffffff ? 2 * V - 7 : 0)) {
        const int b = llb::mass_bits(V);
        const unsigned __int128 unit = static_cast<unsigned __int128>(1) << b, whole = static_cast<unsigned __int128>(1) << 64;
        CHECK(b > 0 && b <= 46);
        CHECK(V * unit < whole);                       // all tokens at the maximum
        CHECK(b == 46 || V * unit * 2 >= whole);       // and no bit less than that takes
    }
    const int V = 262144;
    CHECK(llb::mass_bits(V - 1) == 46 && llb::mass_bits(V) == 45);
    printf("ok\n");
    return 0;
}
