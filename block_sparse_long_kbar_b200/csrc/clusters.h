// How many CTAs a cluster launch takes (host code).
#pragma once

namespace sgqa {

// `want`, or the 8 that are always possible where the current device cannot hold a cluster of more.
// allow: sets the function's attribute for them, true if it could; most: how many such clusters the device
// holds at a time. Both are asked at every launch, since attribute and answer belong to the device (and its
// context), of which a process can have several.
template <class Allow, class Most>
int cluster_ctas(int want, Allow&& allow, Most&& most) {
  return want <= 8 || (allow() && most() > 0) ? want : 8;
}

}  // namespace sgqa
