// Host program of tests/test_draw_grid_host.py: walks the borders of the
// draw's bins. Prints one line per grid; a wrong border is an exit status.
#include <cmath>
#include <cstdio>
#include <cstdlib>

#include "draw_grid.hpp"

int main(int argc, char** argv) {
  const double T = static_cast<double>(std::strtof(argv[1], nullptr));
  const float most = INFINITY;
  const float refs[] = {0.0f, -0.0f, 1.0f, -3.5f, 1e-38f, -1e-38f, 1e-44f, -1e-44f, static_cast<float>(100.0 * T),
                        static_cast<float>(-1e5 * T), 3e38f};
  const int bins[] = {0, 1, 2, 700, vsv::kBase - 2, vsv::kBase - 1, vsv::kBase, vsv::kBase + 1, vsv::kBase + 2, 3000, vsv::kBins - 1};
  for (float ref : refs) {
    for (double per : {32.0, 64.0}) {
      bool far;
      const vsv::Grid g = vsv::Grid::around(ref, T, per, far);
      std::printf("T %g ref %g per %g%s\n", T, ref, per, far ? " far" : "");
      std::fflush(stdout);
      if (far) continue;
      for (int b : bins) {
        const float x = g.least_in(b);
        if (!g.reaches(x, b)) return 2;
        const float below = std::nextafterf(x, -most);
        if (below > -most && below < x && g.reaches(below, b)) return 3;
      }
    }
  }
  return 0;
}
