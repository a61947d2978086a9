// Irreps strings ("64x0e+64x1o"): the parser shared by the convolution plan and the node
// feature plan (host side).
#pragma once
#include <cstdlib>
#include <string>
#include <vector>

#include "../../include/tpconv.h"
#include "internal.h"

namespace tpc {

constexpr int kMaxOrder = 3;  // largest irrep order l

// One irrep block of a node row: mul channels of order l, first element `offset`.
struct Block {
  int mul, l, parity, offset;
};

inline tpconv_status parse_irreps(const char* s, std::vector<Block>& out) {
  if (!s) return TPCONV_ERR_INVALID_ARG;
  out.clear();
  std::string str(s);
  size_t pos = 0;
  int off = 0;
  if (str.find_first_not_of(" \t") == std::string::npos) return TPCONV_ERR_PARSE;
  while (pos <= str.size()) {
    size_t plus = str.find('+', pos);
    std::string tok = str.substr(pos, plus == std::string::npos ? std::string::npos : plus - pos);
    std::string t;
    for (char ch : tok) if (ch != ' ' && ch != '\t') t.push_back(ch);
    if (t.empty()) return TPCONV_ERR_PARSE;
    long mul = 1;
    size_t xp = t.find('x');
    std::string lp = t;
    if (xp != std::string::npos) {
      std::string ms = t.substr(0, xp);
      if (ms.empty() || ms.find_first_not_of("0123456789") != std::string::npos || ms.size() > 6) return TPCONV_ERR_PARSE;
      mul = std::atol(ms.c_str());
      lp = t.substr(xp + 1);
    }
    if (lp.size() < 2) return TPCONV_ERR_PARSE;
    char par = lp.back();
    std::string ls = lp.substr(0, lp.size() - 1);
    if ((par != 'e' && par != 'o') || ls.empty() || ls.find_first_not_of("0123456789") != std::string::npos || ls.size() > 3)
      return TPCONV_ERR_PARSE;
    long l = std::atol(ls.c_str());
    if (mul <= 0) return TPCONV_ERR_PARSE;
    if (l > kMaxOrder) return TPCONV_ERR_UNSUPPORTED;
    Block b{(int)mul, (int)l, par == 'e' ? 1 : -1, off};
    off += b.mul * (2 * b.l + 1);
    out.push_back(b);
    if (plus == std::string::npos) break;
    pos = plus + 1;
  }
  if ((int)out.size() > MAX_BLOCKS) return TPCONV_ERR_UNSUPPORTED;
  return TPCONV_OK;
}

}  // namespace tpc
